// block_api.hip -- the C ABI declared in include/per_block.h: argument checks and
// launches of the operators of a student that reads tokens.  Nothing here allocates
// device memory or waits for the device.

#include <math.h>

#include <algorithm>
#include <utility>

#include "api_checks.h"
#include "block_internal.h"

namespace {

using namespace per;

// Rows of D values, stride elements apart.
int check_rows2(const void* p, int32_t type, int64_t D, int64_t stride, const char* what) {
  if (!p) return bad("%s is required", what);
  if (misaligned(p, size_of(type))) return bad("%s is not aligned to its type", what);
  if (stride < D || stride > kMaxStride)
    return bad("%s has a stride of %lld, below its %lld columns or too large", what,
               (long long)stride, (long long)D);
  return PER_OK;
}

int check_embed(int64_t N, int64_t V, int64_t D) {
  if (N < 0 || N > PER_MAX_TOKENS) return bad("N %lld outside [0, 2^28]", (long long)N);
  if (V < 1 || V > PER_MAX_VOCAB) return bad("V %lld outside [1, 2^24]", (long long)V);
  if (D < 1 || D > PER_MAX_ROW_DIM) return bad("D %lld outside [1, 2^20]", (long long)D);
  return PER_OK;
}
int check_tokens(int64_t N, const void* tokens, int32_t bytes) {
  if (bytes != 4 && bytes != 8) return bad("token_bytes %d is neither 4 nor 8", (int)bytes);
  if (N == 0) return PER_OK;
  if (!tokens) return bad("tokens are required");
  if (misaligned(tokens, bytes)) return bad("tokens are not aligned to their type");
  return PER_OK;
}

int check_norm(int64_t N, int64_t D, int32_t type) {
  if (N < 0 || N > kMaxGrid) return bad("N %lld outside [0, 2^31)", (long long)N);
  if (D < 1 || D > PER_MAX_ROW_DIM) return bad("D %lld outside [1, 2^20]", (long long)D);
  if (!type_ok(type)) return bad("type %d is none", (int)type);
  return PER_OK;
}
int check_affine(const void* p, int32_t affine_type, int32_t type, const char* what) {
  if (!p) return PER_OK;
  if (affine_type != PER_F32 && affine_type != type)
    return bad("%s is neither f32 nor of the type of x", what);
  if (misaligned(p, size_of(affine_type))) return bad("%s is not aligned to its type", what);
  return PER_OK;
}

int check_delta(DeltaArgs& a, int64_t B, int64_t T, int64_t H, int64_t HK, int64_t DK, int64_t DV,
                int32_t type) {
  if (B < 0 || T < 0 || B > kMaxGrid || T > kMaxGrid - PER_DELTA_CHUNK)
    return bad("B or T is negative or too large");
  if (H < 1 || H > 65535 || HK < 1 || H % HK != 0)
    return bad("H %lld outside [1, 2^16), or HK %lld does not divide it", (long long)H,
               (long long)HK);
  if (DK < 1 || DK > PER_DELTA_MAX_DK) return bad("DK %lld outside [1, 128]", (long long)DK);
  if (DV < 1 || DV > PER_DELTA_MAX_DV) return bad("DV %lld outside [1, 256]", (long long)DV);
  if (!type_ok(type)) return bad("type %d is none", (int)type);
  const int64_t chunks = (T + PER_DELTA_CHUNK - 1) / PER_DELTA_CHUNK;
  if (B * H > kMaxGrid / 4 || (B > 0 && chunks > kMaxGrid / (B * H)))
    return bad("B * T * H is too large");
  a = DeltaArgs{};
  a.B = B;
  a.T = T;
  a.H = (int)H;
  a.HK = (int)HK;
  a.DK = (int)DK;
  a.DV = (int)DV;
  a.chunks = chunks;
  return PER_OK;
}
// A chunk's rows lie within 2^31 bytes, so that places in them are 32-bit offsets.
constexpr int64_t kMaxStep = 1 << 23;

// An array of sequences [B x T x H] of rows of D values.  An output's rows must not
// overlap: by rising stride, each dimension steps past the extent of those before.
int check_seq(Seq& to, const per_seq& s, int32_t type, int64_t B, int64_t T, int64_t H, int64_t D,
              bool output, const char* what) {
  if (!s.p) return bad("%s is required", what);
  if (misaligned(s.p, size_of(type))) return bad("%s is not aligned to its type", what);
  if (s.sb < 0 || s.st < 0 || s.sh < 0 || s.sb > kMaxStride || s.st > kMaxStride ||
      s.sh > kMaxStride)
    return bad("%s has a stride that is negative or too large", what);
  if (T > 1 && s.st > kMaxStep)
    return bad("%s has steps %lld elements apart, more than 2^23", what, (long long)s.st);
  if (output) {
    std::pair<int64_t, int64_t> dims[3] = {{s.sb, B}, {s.st, T}, {s.sh, H}};
    std::sort(dims, dims + 3);
    int64_t extent = D;
    for (const auto& d : dims) {
      if (d.second <= 1) continue;
      if (d.first < extent) return bad("%s has rows that overlap", what);
      if (d.second > (int64_t(1) << 60) / d.first) return bad("%s is too large", what);
      extent += (d.second - 1) * d.first;
    }
  }
  to = Seq{s.p, s.sb, T > 1 ? s.st : D, s.sh};
  return PER_OK;
}

struct Inputs {
  per_seq q, k, v, g, b;
};
int check_inputs(DeltaArgs& a, const Inputs& in, int32_t type) {
  int rc;
  if ((rc = check_seq(a.q, in.q, type, a.B, a.T, a.HK, a.DK, false, "q"))) return rc;
  if ((rc = check_seq(a.k, in.k, type, a.B, a.T, a.HK, a.DK, false, "k"))) return rc;
  if ((rc = check_seq(a.v, in.v, type, a.B, a.T, a.H, a.DV, false, "v"))) return rc;
  if ((rc = check_seq(a.g, in.g, type, a.B, a.T, a.H, 1, false, "g"))) return rc;
  return check_seq(a.b, in.b, type, a.B, a.T, a.H, 1, false, "b");
}
int check_scale(double scale, const char* what) {
  if (!isfinite(scale) || !isfinite((float)scale)) return bad("%s is not finite in f32", what);
  return PER_OK;
}

}  // namespace

int per_embed_forward(int64_t N, int64_t V, int64_t D, const void* d_tokens, int32_t token_bytes,
                      const void* d_table, int32_t table_type, int64_t table_stride, double scale,
                      void* d_out, int32_t out_type, int64_t out_stride, hipStream_t stream) {
  int rc = check_embed(N, V, D);
  if (rc) return rc;
  if (!type_ok(table_type) || !type_ok(out_type)) return bad("type is none");
  if ((rc = check_tokens(N, d_tokens, token_bytes))) return rc;
  if ((rc = check_scale(scale, "scale"))) return rc;
  if (N == 0) return api_ok();
  if ((rc = check_rows2(d_table, table_type, D, table_stride, "table"))) return rc;
  if ((rc = check_rows2(d_out, out_type, D, out_stride, "out"))) return rc;
  EmbedArgs a = {};
  a.N = N;
  a.V = V;
  a.D = D;
  a.tokens = d_tokens;
  a.token_bytes = token_bytes;
  a.src = d_table;
  a.src_stride = table_stride;
  a.dst = d_out;
  a.dst_stride = out_stride;
  a.scale = (float)scale;
  return run("per_embed_forward",
             [&] { return launch_embed_forward(a, table_type, out_type, stream); });
}

int per_embed_workspace_bytes(int64_t N, int64_t V, int64_t D, size_t* out) {
  const int rc = check_embed(N, V, D);
  if (rc) return rc;
  if (!out) return bad("out is NULL");
  *out = embed_workspace(N, V, D, nullptr, nullptr);
  return api_ok();
}

int per_embed_backward(int64_t N, int64_t V, int64_t D, const void* d_tokens, int32_t token_bytes,
                       const void* d_dout, int32_t dout_type, int64_t dout_stride, double scale,
                       int32_t accumulate, void* d_grad, int32_t grad_type, int64_t grad_stride,
                       void* d_ws, size_t ws_bytes, hipStream_t stream) {
  int rc = check_embed(N, V, D);
  if (rc) return rc;
  if (!type_ok(dout_type) || !type_ok(grad_type)) return bad("type is none");
  if ((rc = check_tokens(N, d_tokens, token_bytes))) return rc;
  if ((rc = check_scale(scale, "scale"))) return rc;
  if (N > 0 && (rc = check_rows2(d_dout, dout_type, D, dout_stride, "dout"))) return rc;
  if ((rc = check_rows2(d_grad, grad_type, D, grad_stride, "grad"))) return rc;
  if ((rc = check_ws(d_ws, ws_bytes, embed_workspace(N, V, D, nullptr, nullptr)))) return rc;
  EmbedArgs a = {};
  a.N = N;
  a.V = V;
  a.D = D;
  a.tokens = d_tokens;
  a.token_bytes = token_bytes;
  a.src = d_dout;
  a.src_stride = dout_stride;
  a.dst = d_grad;
  a.dst_stride = grad_stride;
  a.scale = (float)scale;
  a.accumulate = accumulate != 0;
  embed_workspace(N, V, D, &a, d_ws);
  return run("per_embed_backward",
             [&] { return launch_embed_backward(a, dout_type, grad_type, stream); });
}

int per_norm_forward(int64_t N, int64_t D, int32_t type, const void* d_x, int64_t x_stride,
                     const void* d_weight, const void* d_bias, int32_t affine_type, double eps,
                     void* d_y, int64_t y_stride, float* d_stats, hipStream_t stream) {
  int rc = check_norm(N, D, type);
  if (rc) return rc;
  if (!(eps >= 0.0) || !isfinite((float)eps)) return bad("eps outside [0, infinity)");
  if ((rc = check_affine(d_weight, affine_type, type, "weight"))) return rc;
  if ((rc = check_affine(d_bias, affine_type, type, "bias"))) return rc;
  if (misaligned(d_stats, 4)) return bad("stats are not aligned to their type");
  if (N == 0) return api_ok();
  if ((rc = check_rows2(d_x, type, D, x_stride, "x"))) return rc;
  if ((rc = check_rows2(d_y, type, D, y_stride, "y"))) return rc;
  if (d_y == d_x && y_stride != x_stride) return bad("y in place of x has another stride");
  NormArgs a = {};
  a.N = N;
  a.D = (uint32_t)D;
  a.x = d_x;
  a.xs = x_stride;
  a.weight = d_weight;
  a.bias = d_bias;
  a.affine_f32 = affine_type == PER_F32;
  a.eps = (float)eps;
  a.y = d_y;
  a.ys = y_stride;
  a.stats = d_stats;
  return run("per_norm_forward", [&] { return launch_norm_forward(a, type, stream); });
}

int per_norm_workspace_bytes(int64_t N, int64_t D, int32_t type, size_t* out) {
  const int rc = check_norm(N, D, type);
  if (rc) return rc;
  if (!out) return bad("out is NULL");
  *out = norm_workspace(N, D, type, nullptr, nullptr);
  return api_ok();
}

int per_norm_backward(int64_t N, int64_t D, int32_t type, const void* d_x, int64_t x_stride,
                      const float* d_stats, const void* d_dy, int64_t dy_stride,
                      const void* d_weight, int32_t affine_type, void* d_dx, int64_t dx_stride,
                      float* d_dweight, float* d_dbias, void* d_ws, size_t ws_bytes,
                      hipStream_t stream) {
  int rc = check_norm(N, D, type);
  if (rc) return rc;
  if ((rc = check_affine(d_weight, affine_type, type, "weight"))) return rc;
  if (misaligned(d_dweight, 4) || misaligned(d_dbias, 4))
    return bad("dweight or dbias is not aligned to its type");
  if (N > 0) {
    if ((rc = check_rows2(d_x, type, D, x_stride, "x"))) return rc;
    if ((rc = check_rows2(d_dy, type, D, dy_stride, "dy"))) return rc;
    if ((rc = check_rows2(d_dx, type, D, dx_stride, "dx"))) return rc;
    if (d_dx == d_dy && dx_stride != dy_stride) return bad("dx in place of dy has another stride");
    if (!d_stats || misaligned(d_stats, 4)) return bad("stats are required, 4-byte aligned");
  }
  if ((rc = check_ws(d_ws, ws_bytes, norm_workspace(N, D, type, nullptr, nullptr)))) return rc;
  NormArgs a = {};
  a.N = N;
  a.D = (uint32_t)D;
  a.x = d_x;
  a.xs = x_stride;
  a.stats = const_cast<float*>(d_stats);
  a.dy = d_dy;
  a.dys = dy_stride;
  a.weight = d_weight;
  a.affine_f32 = affine_type == PER_F32;
  a.y = d_dx;
  a.ys = dx_stride;
  a.dweight = d_dweight;
  a.dbias = d_dbias;
  norm_workspace(N, D, type, &a, d_ws);
  return run("per_norm_backward", [&] { return launch_norm_backward(a, type, stream); });
}

int per_delta_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t HK, int64_t DK, int64_t DV,
                              int32_t type, int32_t backward, size_t* out) {
  DeltaArgs a;
  const int rc = check_delta(a, B, T, H, HK, DK, DV, type);
  if (rc) return rc;
  if (!out) return bad("out is NULL");
  *out = delta_workspace(B, T, H, DK, DV, type, backward != 0, nullptr, nullptr);
  return api_ok();
}

int per_delta_forward(int64_t B, int64_t T, int64_t H, int64_t HK, int64_t DK, int64_t DV,
                      int32_t type, per_seq q, per_seq k, per_seq v, per_seq g, per_seq b,
                      const uint8_t* d_reset, const int64_t* d_length, const float* d_s0,
                      double scale, per_seq o, float* d_s_last, float* d_carries, void* d_ws,
                      size_t ws_bytes, hipStream_t stream) {
  DeltaArgs a;
  int rc = check_delta(a, B, T, H, HK, DK, DV, type);
  if (rc) return rc;
  if ((rc = check_scale(scale, "scale"))) return rc;
  if (B == 0) return api_ok();
  if (T > 0) {
    if ((rc = check_inputs(a, {q, k, v, g, b}, type))) return rc;
    if ((rc = check_seq(a.o, o, type, B, T, H, DV, true, "o"))) return rc;
  }
  if (misaligned(d_length, 8) || misaligned(d_s0, 4) || misaligned(d_s_last, 4) ||
      misaligned(d_carries, 4))
    return bad("length, s0, s_last or carries is not aligned to its type");
  if ((rc = check_ws(d_ws, ws_bytes, delta_workspace(B, T, H, DK, DV, type, false, nullptr, nullptr))))
    return rc;
  a.reset = d_reset;
  a.length = d_length;
  a.s0 = d_s0;
  a.s_last = d_s_last;
  a.carries = d_carries;
  a.scale = (float)scale;
  delta_workspace(B, T, H, DK, DV, type, false, &a, d_ws);
  return run("per_delta_forward", [&] { return launch_delta_forward(a, type, stream); });
}

int per_delta_backward(int64_t B, int64_t T, int64_t H, int64_t HK, int64_t DK, int64_t DV,
                       int32_t type, per_seq q, per_seq k, per_seq v, per_seq g, per_seq b,
                       const uint8_t* d_reset, const int64_t* d_length, const float* d_carries,
                       per_seq d_o, const float* d_ds_last, double scale, per_seq dq, per_seq dk,
                       per_seq dv, per_seq dg, per_seq db, float* d_ds0, void* d_ws,
                       size_t ws_bytes, hipStream_t stream) {
  DeltaArgs a;
  int rc = check_delta(a, B, T, H, HK, DK, DV, type);
  if (rc) return rc;
  if ((rc = check_scale(scale, "scale"))) return rc;
  if (B == 0) return api_ok();
  if (T > 0) {
    if ((rc = check_inputs(a, {q, k, v, g, b}, type))) return rc;
    if ((rc = check_seq(a.o, d_o, type, B, T, H, DV, false, "do"))) return rc;
    if ((rc = check_seq(a.dq, dq, type, B, T, HK, DK, true, "dq"))) return rc;
    if ((rc = check_seq(a.dk, dk, type, B, T, HK, DK, true, "dk"))) return rc;
    if ((rc = check_seq(a.dv, dv, type, B, T, H, DV, true, "dv"))) return rc;
    if ((rc = check_seq(a.dg, dg, type, B, T, H, 1, true, "dg"))) return rc;
    if ((rc = check_seq(a.db, db, type, B, T, H, 1, true, "db"))) return rc;
    if (!d_carries) return bad("carries are required");
  }
  if (misaligned(d_length, 8) || misaligned(d_ds_last, 4) || misaligned(d_ds0, 4) ||
      misaligned(d_carries, 4))
    return bad("length, ds_last, ds0 or carries is not aligned to its type");
  if ((rc = check_ws(d_ws, ws_bytes, delta_workspace(B, T, H, DK, DV, type, true, nullptr, nullptr))))
    return rc;
  a.reset = d_reset;
  a.length = d_length;
  a.s0 = d_ds_last;
  a.s_last = d_ds0;
  a.carries = const_cast<float*>(d_carries);
  a.scale = (float)scale;
  delta_workspace(B, T, H, DK, DV, type, true, &a, d_ws);
  return run("per_delta_backward", [&] { return launch_delta_backward(a, type, stream); });
}

int per_delta_step(int64_t B, int64_t H, int64_t HK, int64_t DK, int64_t DV, int32_t type,
                   per_seq q, per_seq k, per_seq v, per_seq g, per_seq b, const uint8_t* d_reset,
                   const float* d_s, double scale, float* d_s_out, per_seq o, hipStream_t stream) {
  DeltaArgs a;
  int rc = check_delta(a, B, 1, H, HK, DK, DV, type);
  if (rc) return rc;
  if ((rc = check_scale(scale, "scale"))) return rc;
  if (B == 0) return api_ok();
  if ((rc = check_inputs(a, {q, k, v, g, b}, type))) return rc;
  if ((rc = check_seq(a.o, o, type, B, 1, H, DV, true, "o"))) return rc;
  if (!d_s || !d_s_out) return bad("s and s_out are required");
  if (misaligned(d_s, 4) || misaligned(d_s_out, 4)) return bad("s or s_out is not aligned");
  a.reset = d_reset;
  a.s0 = d_s;
  a.s_last = d_s_out;
  a.scale = (float)scale;
  return run("per_delta_step", [&] { return launch_delta_step(a, type, stream); });
}
