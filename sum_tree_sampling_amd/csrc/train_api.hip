// train_api.hip -- the C ABI declared in include/per_train.h: argument checks
// and launches of the sequence operators.  Nothing here allocates device
// memory or waits for the device.

#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include "../../include/per_train.h"
#include "train_internal.h"

namespace {

__attribute__((format(printf, 1, 2))) int bad(const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return per::api_fail(PER_EINVAL, buf);
}

thread_local per::Launches g_launches;

// Runs a call's launches, once to count and then in earnest.
template <typename F>
int run(const char* what, F launch) {
  g_launches.counting = true;
  g_launches.items = 0;
  hipError_t e = launch();
  g_launches.counting = false;
  if (e == hipSuccess && g_launches.items >> 32)
    return bad("%s would take %llu work-items in one launch, 2^32 or more: call it in pieces", what,
               (unsigned long long)g_launches.items);
  if (e == hipSuccess) e = launch();
  if (e == hipSuccess) return per::api_ok();
  char buf[256];
  snprintf(buf, sizeof buf, "%s: %s", what, hipGetErrorString(e));
  return per::api_fail(PER_EHIP, buf);
}

bool type_ok(int32_t t) { return t == PER_F32 || t == PER_BF16 || t == PER_F16; }
int size_of(int32_t t) { return t == PER_F32 ? 4 : 2; }

bool misaligned(const void* p, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) != 0;
}

constexpr int64_t kMaxGrid = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxStride = int64_t(1) << 40;

// What the three calls of the row store have in common.
int check_rows(per::RowsArgs& a, int64_t capacity, int64_t dim, int32_t format, int32_t group,
               uint8_t* codes, int64_t cs, float* scales, int64_t ss, int32_t type, int64_t stride) {
  if (capacity < 1 || capacity > PER_MAX_CAPACITY)
    return bad("capacity %lld outside [1, 2^30]", (long long)capacity);
  if (dim < 1 || dim > PER_MAX_ROW_DIM)
    return bad("dim %lld outside [1, 2^20]", (long long)dim);
  if (format != PER_E4M3 && format != PER_I8) return bad("format %d is none", (int)format);
  if (group != 0 && group != 32 && group != 64 && group != 128)
    return bad("group %d is none of 0, 32, 64, 128", (int)group);
  if (!type_ok(type)) return bad("type %d is none", (int)type);
  if (!codes || !scales) return bad("codes and scales are required");
  if (misaligned(scales, 4)) return bad("scales must be 4-byte aligned");
  const int64_t ng = group == 0 ? 1 : (dim + group - 1) / group;
  if (cs < dim || cs > kMaxStride) return bad("codes_stride %lld below dim", (long long)cs);
  if (ss < ng || ss > kMaxStride)
    return bad("scales_stride %lld below the %lld scales of a row", (long long)ss, (long long)ng);
  if (stride < dim || stride > kMaxStride)
    return bad("row stride %lld below dim", (long long)stride);
  a = per::RowsArgs{};
  a.codes = codes;
  a.scales = scales;
  a.cs = cs;
  a.ss = ss;
  a.capacity = capacity;
  a.stride = stride;
  a.dim = (uint32_t)dim;
  a.window = 1;
  a.lg_group = group == 0 ? -1 : group == 32 ? 2 : group == 64 ? 3 : 4;
  return PER_OK;
}

int check_scan(int64_t B, int64_t T, int64_t D, int32_t type) {
  if (B < 0 || T < 0 || D < 1) return bad("B, T or D is negative, or D is 0");
  if (!type_ok(type)) return bad("type %d is none", (int)type);
  // bounds every product of sizes below
  if (B > kMaxGrid || T > (int64_t(1) << 40) || D > (int64_t(1) << 31))
    return bad("B, T or D is too large");
  if (B > 0 && per::scan_blocks(B, T, D) > kMaxGrid) return bad("B * D is too large");
  return PER_OK;
}

int check_view(const void* p, int32_t type, int64_t sb, int64_t st, const char* what) {
  if (!p) return bad("%s is required", what);
  if (misaligned(p, size_of(type))) return bad("%s is not aligned to its type", what);
  if (sb < 0 || st < 0 || sb > kMaxStride || st > kMaxStride)
    return bad("%s has a stride that is negative or too large", what);
  return PER_OK;
}

// An output's steps and sequences must not overlap: rows of D channels, the
// smaller stride's whole extent within the larger one.
int check_out_view(const void* p, int32_t type, int64_t B, int64_t T, int64_t D, int64_t sb,
                   int64_t st, const char* what) {
  const int rc = check_view(p, type, sb, st, what);
  if (rc) return rc;
  const bool t_inner = T <= 1 || (st >= D && (B <= 1 || sb >= (T - 1) * st + D));
  const bool b_inner = B <= 1 || (sb >= D && (T <= 1 || st >= (B - 1) * sb + D));
  if ((T <= 1 && B > 1 && sb < D) || !(t_inner || b_inner))
    return bad("%s has rows that overlap", what);
  return PER_OK;
}

int check_ws(const void* ws, size_t have, size_t need) {
  if (need == 0) return PER_OK;
  if (!ws) return bad("a workspace of %zu bytes is required", need);
  if (misaligned(ws, 16)) return bad("the workspace must be 16-byte aligned");
  if (have < need) {
    char buf[128];
    snprintf(buf, sizeof buf, "workspace of %zu bytes, %zu are needed", have, need);
    return per::api_fail(PER_ENOSPC, buf);
  }
  return PER_OK;
}

int check_distill(per::DistillArgs& a, int64_t N, int64_t V, int64_t K, int32_t type,
                  const void* z, int64_t stride, const int32_t* tidx, const void* t,
                  int32_t t_type, const float* tlse, double tau) {
  if (N < 0 || N > kMaxGrid) return bad("N %lld outside [0, 2^31)", (long long)N);
  if (V < 1 || V > PER_MAX_VOCAB) return bad("V %lld outside [1, 2^24]", (long long)V);
  if (K < 1 || K > PER_MAX_TOP) return bad("K %lld outside [1, 1024]", (long long)K);
  if (!type_ok(type) || !type_ok(t_type)) return bad("type is none");
  if (!(tau >= 0x1p-20 && tau <= 0x1p6)) return bad("temperature outside [2^-20, 2^6]");
  if (stride < V || stride > kMaxStride) return bad("logits' stride %lld below V", (long long)stride);
  if (N == 0) return PER_OK;
  if (!z || !tidx || !t) return bad("logits, token indices and teacher logits are required");
  if (misaligned(z, size_of(type)) || misaligned(tidx, 4) || misaligned(t, size_of(t_type)) ||
      misaligned(tlse, 4))
    return bad("an input is not aligned to its type");
  if (N * (int64_t)per::distill_splits(N, V, type) > kMaxGrid) return bad("N * V is too large");
  a = per::DistillArgs{};
  a.N = N;
  a.V = V;
  a.K = (int)K;
  a.z = z;
  a.stride = stride;
  a.tidx = tidx;
  a.t = t;
  a.t_type = t_type;
  a.tlse = tlse;
  a.inv_tau = 1.0 / tau;
  a.c = (float)(1.44269504088896340736 / tau);
  a.tau = (float)tau;
  a.splits = per::distill_splits(N, V, type);
  return PER_OK;
}

// Workspace of rows taken in parts: the teacher's sums of each row, each part's
// statistics, and what per_distill saves between its passes.
struct DistillSpace {
  size_t part, saved, total;
};
DistillSpace distill_space(int64_t N, int64_t V, int64_t K, int32_t type) {
  DistillSpace s = {0, 0, 0};
  if (per::distill_small(N, V, type)) return s;
  s.part = (size_t)N * sizeof(per::Teacher);
  s.saved = s.part + (size_t)N * per::distill_splits(N, V, type) * 24;
  s.total = s.saved + (size_t)N * (size_t)(4 + K) * 4;
  return s;
}
void set_space(per::DistillArgs& a, void* ws, int32_t type) {
  const DistillSpace s = distill_space(a.N, a.V, a.K, type);
  char* base = static_cast<char*>(ws);
  a.teacher = reinterpret_cast<per::Teacher*>(base);
  a.part = base + s.part;
  a.saved = reinterpret_cast<float*>(base + s.saved);
}

int check_grad(const void* grad, int64_t stride, int32_t type, int64_t V, const void* z,
               int64_t z_stride) {
  if (!grad) return bad("grad is required");
  if (misaligned(grad, size_of(type))) return bad("grad is not aligned to its type");
  if (stride < V || stride > kMaxStride) return bad("grad's stride %lld below V", (long long)stride);
  if (grad == z && stride != z_stride) return bad("grad in place of logits has another stride");
  return PER_OK;
}

}  // namespace

per::Launches& per::launches() { return g_launches; }

int per_rows_write(int64_t capacity, int64_t dim, int32_t format, int32_t group, uint8_t* d_codes,
                   int64_t codes_stride, float* d_scales, int64_t scales_stride, int64_t count,
                   int64_t first, const void* d_src, int32_t type, int64_t src_stride,
                   hipStream_t stream) {
  per::RowsArgs a;
  const int rc = check_rows(a, capacity, dim, format, group, d_codes, codes_stride, d_scales,
                            scales_stride, type, src_stride);
  if (rc) return rc;
  if (count < 0 || count > capacity)
    return bad("count %lld outside [0, capacity]", (long long)count);
  if (first < 0 || first >= capacity)
    return bad("first %lld outside [0, capacity)", (long long)first);
  if (count == 0) return per::api_ok();
  if (!d_src) return bad("src is required");
  if (misaligned(d_src, size_of(type))) return bad("src is not aligned to its type");
  a.src = d_src;
  a.first = first;
  a.rows = (uint32_t)count;
  return run("per_rows_write", [&] { return per::launch_rows_write(a, type, format, stream); });
}

int per_rows_write_at(int64_t capacity, int64_t dim, int32_t format, int32_t group,
                      uint8_t* d_codes, int64_t codes_stride, float* d_scales,
                      int64_t scales_stride, int64_t count, const int64_t* d_slots,
                      uint32_t* d_claims, const void* d_src, int32_t type, int64_t src_stride,
                      hipStream_t stream) {
  per::RowsArgs a;
  const int rc = check_rows(a, capacity, dim, format, group, d_codes, codes_stride, d_scales,
                            scales_stride, type, src_stride);
  if (rc) return rc;
  if (count < 0 || count > kMaxGrid) return bad("count %lld outside [0, 2^31)", (long long)count);
  if (count == 0) return per::api_ok();
  if (!d_src || !d_slots || !d_claims) return bad("src, slots and claims are required");
  if (misaligned(d_src, size_of(type)) || misaligned(d_slots, 8) || misaligned(d_claims, 4))
    return bad("src, slots or claims is not aligned to its type");
  a.src = d_src;
  a.slots = d_slots;
  a.claims = d_claims;
  a.rows = (uint32_t)count;
  return run("per_rows_write_at", [&] { return per::launch_rows_write(a, type, format, stream); });
}

int per_rows_read(int64_t capacity, int64_t dim, int32_t format, int32_t group,
                  const uint8_t* d_codes, int64_t codes_stride, const float* d_scales,
                  int64_t scales_stride, int64_t B, const int64_t* d_idx, int64_t window,
                  void* d_out, int32_t type, int64_t out_stride, hipStream_t stream) {
  per::RowsArgs a;
  const int rc = check_rows(a, capacity, dim, format, group, const_cast<uint8_t*>(d_codes),
                            codes_stride, const_cast<float*>(d_scales), scales_stride, type,
                            out_stride);
  if (rc) return rc;
  if (B < 0 || window < 1 || B > kMaxGrid || window > kMaxGrid || B * window > kMaxGrid)
    return bad("B %lld, window %lld: B * window outside [0, 2^31), or window below 1",
               (long long)B, (long long)window);
  if (B == 0) return per::api_ok();
  if (!d_idx || !d_out) return bad("idx and out are required");
  if (misaligned(d_idx, 8) || misaligned(d_out, size_of(type)))
    return bad("idx or out is not aligned to its type");
  a.slots = d_idx;
  a.out = d_out;
  a.window = (uint32_t)window;
  a.rows = (uint32_t)(B * window);
  return run("per_rows_read", [&] { return per::launch_rows_read(a, type, format, stream); });
}

int per_scan_workspace_bytes(int64_t B, int64_t T, int64_t D, size_t* out) {
  const int rc = check_scan(B, T, D, PER_F32);
  if (rc) return rc;
  if (!out) return bad("out is NULL");
  *out = B > 0 ? per::scan_workspace(B, T, D) : 0;
  return per::api_ok();
}

int per_scan_forward(int64_t B, int64_t T, int64_t D, int32_t type, const void* d_x, int64_t x_sb,
                     int64_t x_st, const void* d_g, int64_t g_sb, int64_t g_st,
                     const uint8_t* d_reset, const int64_t* d_length, const float* d_h0, void* d_y,
                     int64_t y_sb, int64_t y_st, float* d_h_last, float* d_carries, void* d_ws,
                     size_t ws_bytes, hipStream_t stream) {
  int rc = check_scan(B, T, D, type);
  if (rc) return rc;
  if (B == 0) return per::api_ok();
  if (T > 0) {
    if ((rc = check_view(d_x, type, x_sb, x_st, "x"))) return rc;
    if ((rc = check_view(d_g, type, g_sb, g_st, "g"))) return rc;
    if ((rc = check_out_view(d_y, type, B, T, D, y_sb, y_st, "y"))) return rc;
  }
  if (misaligned(d_length, 8) || misaligned(d_h0, 4) || misaligned(d_h_last, 4) ||
      misaligned(d_carries, 4))
    return bad("length, h0, h_last or carries is not aligned to its type");
  if ((rc = check_ws(d_ws, ws_bytes, per::scan_workspace(B, T, D)))) return rc;
  per::ScanArgs a = {};
  a.B = B;
  a.T = T;
  a.D = D;
  a.x = d_x;
  a.x_sb = x_sb;
  a.x_st = x_st;
  a.g = d_g;
  a.g_sb = g_sb;
  a.g_st = g_st;
  a.y = d_y;
  a.y_sb = y_sb;
  a.y_st = y_st;
  a.reset = d_reset;
  a.length = d_length;
  a.h0 = d_h0;
  a.h_last = d_h_last;
  a.carries = d_carries;
  a.agg = static_cast<float*>(d_ws);
  return run("per_scan_forward", [&] { return per::launch_scan_forward(a, type, stream); });
}

int per_scan_backward(int64_t B, int64_t T, int64_t D, int32_t type, const void* d_x, int64_t x_sb,
                      int64_t x_st, const void* d_g, int64_t g_sb, int64_t g_st,
                      const uint8_t* d_reset, const int64_t* d_length, const float* d_carries,
                      const void* d_dy, int64_t dy_sb, int64_t dy_st, const float* d_dh_last,
                      void* d_dx, int64_t dx_sb, int64_t dx_st, void* d_dg, int64_t dg_sb,
                      int64_t dg_st, float* d_dh0, void* d_ws, size_t ws_bytes,
                      hipStream_t stream) {
  int rc = check_scan(B, T, D, type);
  if (rc) return rc;
  if (B == 0) return per::api_ok();
  if (T > 0) {
    if ((rc = check_view(d_x, type, x_sb, x_st, "x"))) return rc;
    if ((rc = check_view(d_g, type, g_sb, g_st, "g"))) return rc;
    if ((rc = check_view(d_dy, type, dy_sb, dy_st, "dy"))) return rc;
    if ((rc = check_out_view(d_dx, type, B, T, D, dx_sb, dx_st, "dx"))) return rc;
    if ((rc = check_out_view(d_dg, type, B, T, D, dg_sb, dg_st, "dg"))) return rc;
    if (!d_carries) return bad("carries are required");
  }
  if (misaligned(d_length, 8) || misaligned(d_dh_last, 4) || misaligned(d_dh0, 4) ||
      misaligned(d_carries, 4))
    return bad("length, dh_last, dh0 or carries is not aligned to its type");
  if ((rc = check_ws(d_ws, ws_bytes, per::scan_workspace(B, T, D)))) return rc;
  per::ScanArgs a = {};
  a.B = B;
  a.T = T;
  a.D = D;
  a.x = d_x;
  a.x_sb = x_sb;
  a.x_st = x_st;
  a.g = d_g;
  a.g_sb = g_sb;
  a.g_st = g_st;
  a.dy = d_dy;
  a.dy_sb = dy_sb;
  a.dy_st = dy_st;
  a.dx = d_dx;
  a.dx_sb = dx_sb;
  a.dx_st = dx_st;
  a.dg = d_dg;
  a.dg_sb = dg_sb;
  a.dg_st = dg_st;
  a.reset = d_reset;
  a.length = d_length;
  a.carries = const_cast<float*>(d_carries);
  a.dh_last = d_dh_last;
  a.dh0 = d_dh0;
  a.agg = static_cast<float*>(d_ws);
  return run("per_scan_backward", [&] { return per::launch_scan_backward(a, type, stream); });
}

int per_scan_step(int64_t B, int64_t D, int32_t type, const void* d_x, int64_t x_stride,
                  const void* d_g, int64_t g_stride, const uint8_t* d_reset, const float* d_h,
                  float* d_h_out, void* d_y, int64_t y_stride, hipStream_t stream) {
  int rc = check_scan(B, 1, D, type);
  if (rc) return rc;
  if (B == 0) return per::api_ok();
  if ((rc = check_view(d_x, type, x_stride, 0, "x"))) return rc;
  if ((rc = check_view(d_g, type, g_stride, 0, "g"))) return rc;
  if ((rc = check_out_view(d_y, type, B, 1, D, y_stride, 0, "y"))) return rc;
  if (!d_h || !d_h_out) return bad("h and h_out are required");
  if (misaligned(d_h, 4) || misaligned(d_h_out, 4)) return bad("h or h_out is not aligned");
  per::StepArgs a = {};
  a.B = B;
  a.D = D;
  a.x = d_x;
  a.x_st = x_stride;
  a.g = d_g;
  a.g_st = g_stride;
  a.y = d_y;
  a.y_st = y_stride;
  a.reset = d_reset;
  a.h = d_h;
  a.h_out = d_h_out;
  return run("per_scan_step", [&] { return per::launch_scan_step(a, type, stream); });
}

int per_distill_workspace_bytes(int64_t N, int64_t V, int64_t K, int32_t type, size_t* out) {
  if (N < 0 || N > kMaxGrid || V < 1 || V > PER_MAX_VOCAB || K < 1 || K > PER_MAX_TOP)
    return bad("N, V or K is out of range");
  if (!type_ok(type)) return bad("type %d is none", (int)type);
  if (!out) return bad("out is NULL");
  *out = N > 0 ? distill_space(N, V, K, type).total : 0;
  return per::api_ok();
}

int per_distill(int64_t N, int64_t V, int64_t K, int32_t type, const void* d_logits,
                int64_t stride, const int32_t* d_tidx, const void* d_tlogit, int32_t tlogit_type,
                const float* d_tlse, double temperature, const float* d_weight, float* d_loss,
                void* d_grad, int64_t grad_stride, void* d_ws, size_t ws_bytes,
                hipStream_t stream) {
  per::DistillArgs a;
  int rc = check_distill(a, N, V, K, type, d_logits, stride, d_tidx, d_tlogit, tlogit_type, d_tlse,
                         temperature);
  if (rc) return rc;
  if (N == 0) return per::api_ok();
  if ((rc = check_grad(d_grad, grad_stride, type, V, d_logits, stride))) return rc;
  if (!d_loss || misaligned(d_loss, 4) || misaligned(d_weight, 4))
    return bad("loss is required, loss and weight 4-byte aligned");
  a.weight = d_weight;
  a.loss = d_loss;
  a.grad = d_grad;
  a.grad_stride = grad_stride;
  if (per::distill_resident(N, V, type))
    return run("per_distill", [&] { return per::launch_distill_fused(a, type, stream); });
  if ((rc = check_ws(d_ws, ws_bytes, distill_space(N, V, K, type).total))) return rc;
  set_space(a, d_ws, type);
  return run("per_distill", [&] {
    const hipError_t e = per::launch_distill_forward(a, type, stream);
    return e == hipSuccess ? per::launch_distill_backward(a, type, stream) : e;
  });
}

int per_distill_forward(int64_t N, int64_t V, int64_t K, int32_t type, const void* d_logits,
                        int64_t stride, const int32_t* d_tidx, const void* d_tlogit,
                        int32_t tlogit_type, const float* d_tlse, double temperature,
                        float* d_loss, float* d_saved, void* d_ws, size_t ws_bytes,
                        hipStream_t stream) {
  per::DistillArgs a;
  int rc = check_distill(a, N, V, K, type, d_logits, stride, d_tidx, d_tlogit, tlogit_type, d_tlse,
                         temperature);
  if (rc) return rc;
  if (N == 0) return per::api_ok();
  if (!d_loss || misaligned(d_loss, 4) || misaligned(d_saved, 4))
    return bad("loss is required, loss and saved 4-byte aligned");
  if ((rc = check_ws(d_ws, ws_bytes, distill_space(N, V, K, type).total))) return rc;
  set_space(a, d_ws, type);
  a.loss = d_loss;
  a.saved = d_saved;
  return run("per_distill_forward", [&] { return per::launch_distill_forward(a, type, stream); });
}

int per_distill_backward(int64_t N, int64_t V, int64_t K, int32_t type, const void* d_logits,
                         int64_t stride, const int32_t* d_tidx, const void* d_tlogit,
                         int32_t tlogit_type, const float* d_tlse, double temperature,
                         const float* d_saved, const float* d_gloss, void* d_grad,
                         int64_t grad_stride, hipStream_t stream) {
  per::DistillArgs a;
  int rc = check_distill(a, N, V, K, type, d_logits, stride, d_tidx, d_tlogit, tlogit_type, d_tlse,
                         temperature);
  if (rc) return rc;
  if (N == 0) return per::api_ok();
  if ((rc = check_grad(d_grad, grad_stride, type, V, d_logits, stride))) return rc;
  if (!d_saved || !d_gloss || misaligned(d_saved, 4) || misaligned(d_gloss, 4))
    return bad("saved and gloss are required, 4-byte aligned");
  a.saved = const_cast<float*>(d_saved);
  a.weight = d_gloss;
  a.grad = d_grad;
  a.grad_stride = grad_stride;
  return run("per_distill_backward", [&] { return per::launch_distill_backward(a, type, stream); });
}
