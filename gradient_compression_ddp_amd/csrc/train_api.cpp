// C ABI of the training-step operators (gc_train.h): argument checks and dispatch.  Every
// check runs on the host before anything is enqueued, so a rejected call touches no memory
// and makes no HIP call.
#include "gc_train.h"

#include <hip/hip_runtime.h>

#include <initializer_list>

#include "gc.h"
#include "internal.hpp"
#include "overlap.hpp"
#include "train_internal.hpp"

namespace {

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 64;
constexpr int64_t kMaxSpan = int64_t(1) << 40;
constexpr int64_t kMaxFeatures = int64_t(1) << 22;   // of a linear layer: its tiles fit a grid

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int64_t elem_size(int dtype) { return dtype == GC_F32 ? 4 : 2; }

int ok() { return gc::report(GC_OK, "%s", ""); }

int launched(hipError_t e, const char* what) {
  if (e == hipSuccess) return ok();
  return gc::report(GC_EHIP, "%s launch: %s", what, hipGetErrorString(e));
}

#define GC_REQUIRE(cond, ...) \
  do {                        \
    if (!(cond)) return gc::report(GC_EINVAL, __VA_ARGS__); \
  } while (0)
#define GC_TRY(call)              \
  do {                            \
    const int st_ = (call);       \
    if (st_ != GC_OK) return st_; \
  } while (0)

int check_shape(int dtype, int64_t rows, int64_t cols) {
  GC_REQUIRE(dtype >= GC_F32 && dtype <= GC_BF16, "unknown dtype %d", dtype);
  GC_REQUIRE(rows >= 0 && rows <= kMaxDim && cols >= 0 && cols <= kMaxDim, "rows and cols must lie in [0, 2^31 - 64]");
  return GC_OK;
}

// A rows x cols matrix at p whose rows start ld elements apart.
int check_matrix(const char* name, const void* p, int64_t ld, int dtype, int64_t rows, int64_t cols) {
  GC_REQUIRE(p && aligned(p, (size_t)elem_size(dtype)), "%s must be non-NULL and aligned to its element", name);
  GC_REQUIRE(ld >= cols, "%s: a row stride of %lld elements is less than its %lld columns", name, (long long)ld, (long long)cols);
  GC_REQUIRE(ld <= kMaxSpan / rows, "%s: rows * stride must be at most 2^40", name);
  return GC_OK;
}

int check_ckpt(const char* name, const void* codes, const void* exps, int64_t rows, int64_t cols) {
  GC_REQUIRE(codes && aligned(codes, 16), "%s codes must be non-NULL and 16-byte aligned", name);
  GC_REQUIRE(exps != nullptr, "%s exponents must be non-NULL", name);
  GC_REQUIRE((cols + 31) / 32 * 32 <= kMaxSpan / rows, "%s: more than 2^40 codes", name);
  return GC_OK;
}

// An optional checkpoint output: both arrays or neither.
int check_pack(const char* name, const void* codes, const void* exps, int64_t rows, int64_t cols) {
  GC_REQUIRE((codes == nullptr) == (exps == nullptr), "%s codes and exponents: both or neither", name);
  return codes ? check_ckpt(name, codes, exps, rows, cols) : GC_OK;
}

int check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return GC_OK;
  if (!ws) return gc::report(GC_EWORKSPACE, "workspace is NULL but %zu bytes are needed", need);
  GC_REQUIRE(aligned(ws, 256), "workspace must be 256-byte aligned");
  if (have < need) return gc::report(GC_EWORKSPACE, "workspace has %zu bytes, needs %zu", have, need);
  return GC_OK;
}

int check_weight_type(int dtype, int wdtype) {
  GC_REQUIRE(wdtype == dtype || wdtype == GC_F32, "weights are of the input's type or fp32");
  return GC_OK;
}

// What a call reads (out: false) and writes.  Threads read up to 8 elements that other threads write in a call on one
// memory, so outputs in place of inputs are refused.
struct Use {
  const char* name;
  gc::Area area;
  bool out;
};
Use use(const char* name, bool out, const void* p, int64_t ld, int dtype, int64_t rows, int64_t cols) {
  const int64_t s = elem_size(dtype);
  return {name, {reinterpret_cast<uintptr_t>(p), cols * s, ld * s, rows}, out};
}
Use use_bytes(const char* name, bool out, const void* p, int64_t n) {
  return {name, {reinterpret_cast<uintptr_t>(p), n, n, 1}, out};
}
int64_t codes_of(int64_t rows, int64_t cols) { return rows * ((cols + 31) / 32 * 32); }

int check_apart(std::initializer_list<Use> uses) {
  for (const Use* a = uses.begin(); a != uses.end(); ++a) {
    for (const Use* b = a + 1; b != uses.end(); ++b)
      GC_REQUIRE(!(a->out || b->out) || !gc::overlap(a->area, b->area), "%s and %s overlap", a->name, b->name);
  }
  return GC_OK;
}

bool f32_ok(const void* p) { return !p || aligned(p, 4); }

hipStream_t to_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

}  // namespace

extern "C" {

int gc_ckpt_pack(int dtype, const void* x, int64_t ldx, int64_t rows, int64_t cols, int8_t* codes, uint8_t* exps,
                 void* stream) {
  GC_TRY(check_shape(dtype, rows, cols));
  if (rows == 0 || cols == 0) return ok();
  GC_TRY(check_matrix("x", x, ldx, dtype, rows, cols));
  GC_TRY(check_ckpt("x", codes, exps, rows, cols));
  GC_TRY(check_apart({use("x", false, x, ldx, dtype, rows, cols), use_bytes("codes", true, codes, codes_of(rows, cols)),
                      use_bytes("exponents", true, exps, codes_of(rows, cols) / 32)}));
  gc::ActFwdArgs a{};
  a.x = x; a.ldx = ldx; a.rows = rows; a.cols = cols;
  a.x_codes = codes; a.x_exps = exps;
  return launched(gc::launch_act_forward(dtype, -1, a, to_stream(stream)), "gc_ckpt_pack");
}

int gc_ckpt_unpack(int dtype, const int8_t* codes, const uint8_t* exps, int64_t rows, int64_t cols, void* out,
                   int64_t ldo, void* stream) {
  GC_TRY(check_shape(dtype, rows, cols));
  if (rows == 0 || cols == 0) return ok();
  GC_TRY(check_ckpt("the checkpoint's", codes, exps, rows, cols));
  GC_TRY(check_matrix("out", out, ldo, dtype, rows, cols));
  GC_TRY(check_apart({use_bytes("codes", false, codes, codes_of(rows, cols)), use("out", true, out, ldo, dtype, rows, cols),
                      use_bytes("exponents", false, exps, codes_of(rows, cols) / 32)}));
  gc::ActBwdArgs a{};
  a.x_codes = codes; a.x_exps = exps; a.rows = rows; a.cols = cols;
  a.dx = out; a.lddx = ldo;
  return launched(gc::launch_act_backward(dtype, -1, a, to_stream(stream)), "gc_ckpt_unpack");
}

int gc_act_forward(int dtype, int kind, const void* x, int64_t ldx, int64_t rows, int64_t cols, void* y, int64_t ldy,
                   int8_t* x_codes, uint8_t* x_exps, int8_t* y_codes, uint8_t* y_exps, void* stream) {
  GC_TRY(check_shape(dtype, rows, cols));
  GC_REQUIRE(kind >= GC_ACT_GELU && kind <= GC_ACT_SILU, "unknown activation %d", kind);
  if (rows == 0 || cols == 0) return ok();
  GC_TRY(check_matrix("x", x, ldx, dtype, rows, cols));
  GC_TRY(check_matrix("y", y, ldy, dtype, rows, cols));
  GC_TRY(check_pack("x", x_codes, x_exps, rows, cols));
  GC_TRY(check_pack("y", y_codes, y_exps, rows, cols));
  GC_TRY(check_apart({use("x", false, x, ldx, dtype, rows, cols), use("y", true, y, ldy, dtype, rows, cols),
                      use_bytes("x's codes", true, x_codes, codes_of(rows, cols)), use_bytes("x's exponents", true, x_exps, codes_of(rows, cols) / 32),
                      use_bytes("y's codes", true, y_codes, codes_of(rows, cols)), use_bytes("y's exponents", true, y_exps, codes_of(rows, cols) / 32)}));
  gc::ActFwdArgs a{};
  a.x = x; a.ldx = ldx; a.rows = rows; a.cols = cols; a.y = y; a.ldy = ldy;
  a.x_codes = x_codes; a.x_exps = x_exps; a.y_codes = y_codes; a.y_exps = y_exps;
  return launched(gc::launch_act_forward(dtype, kind, a, to_stream(stream)), "gc_act_forward");
}

int gc_act_backward(int dtype, int kind, const void* dy, int64_t lddy, const void* x, int64_t ldx, const int8_t* x_codes,
                    const uint8_t* x_exps, int64_t rows, int64_t cols, void* dx, int64_t lddx, void* stream) {
  GC_TRY(check_shape(dtype, rows, cols));
  GC_REQUIRE(kind >= GC_ACT_GELU && kind <= GC_ACT_SILU, "unknown activation %d", kind);
  if (rows == 0 || cols == 0) return ok();
  GC_REQUIRE((x != nullptr) != (x_codes != nullptr), "exactly one of x and its checkpoint");
  GC_TRY(check_matrix("dy", dy, lddy, dtype, rows, cols));
  if (x) GC_TRY(check_matrix("x", x, ldx, dtype, rows, cols));
  else GC_TRY(check_ckpt("x", x_codes, x_exps, rows, cols));
  GC_TRY(check_matrix("dx", dx, lddx, dtype, rows, cols));
  GC_TRY(check_apart({use("dy", false, dy, lddy, dtype, rows, cols), use("dx", true, dx, lddx, dtype, rows, cols),
                      use("x", false, x, ldx, dtype, rows, cols),
                      use_bytes("codes", false, x_codes, codes_of(rows, cols)), use_bytes("exponents", false, x_exps, codes_of(rows, cols) / 32)}));
  gc::ActBwdArgs a{};
  a.dy = dy; a.lddy = lddy; a.x = x; a.ldx = ldx; a.x_codes = x_codes; a.x_exps = x_exps;
  a.rows = rows; a.cols = cols; a.dx = dx; a.lddx = lddx;
  return launched(gc::launch_act_backward(dtype, kind, a, to_stream(stream)), "gc_act_backward");
}

int gc_layernorm_forward(int dtype, const void* x, int64_t ldx, int64_t rows, int64_t cols, int wdtype,
                         const void* weight, const void* bias, float eps, void* y, int64_t ldy, float* mean,
                         float* rstd, int8_t* x_codes, uint8_t* x_exps, int8_t* y_codes, uint8_t* y_exps, void* stream) {
  GC_TRY(check_shape(dtype, rows, cols));
  GC_TRY(check_weight_type(dtype, wdtype));
  GC_REQUIRE(eps >= 0.0f, "eps must be >= 0");
  if (rows == 0) return ok();
  GC_REQUIRE(cols >= 1, "cols must be >= 1");
  GC_TRY(check_matrix("x", x, ldx, dtype, rows, cols));
  GC_TRY(check_matrix("y", y, ldy, dtype, rows, cols));
  GC_REQUIRE(aligned(weight, (size_t)elem_size(wdtype)) && aligned(bias, (size_t)elem_size(wdtype)),
             "weight and bias must be aligned to their element");
  GC_REQUIRE(mean && rstd && f32_ok(mean) && f32_ok(rstd), "mean and rstd must be non-NULL and 4-byte aligned");
  GC_TRY(check_pack("x", x_codes, x_exps, rows, cols));
  GC_TRY(check_pack("y", y_codes, y_exps, rows, cols));
  GC_TRY(check_apart({use("x", false, x, ldx, dtype, rows, cols), use("y", true, y, ldy, dtype, rows, cols),
                      use("weight", false, weight, cols, wdtype, 1, cols), use("bias", false, bias, cols, wdtype, 1, cols),
                      use_bytes("mean", true, mean, rows * 4), use_bytes("rstd", true, rstd, rows * 4),
                      use_bytes("x's codes", true, x_codes, codes_of(rows, cols)), use_bytes("x's exponents", true, x_exps, codes_of(rows, cols) / 32),
                      use_bytes("y's codes", true, y_codes, codes_of(rows, cols)), use_bytes("y's exponents", true, y_exps, codes_of(rows, cols) / 32)}));
  gc::LnFwdArgs a{};
  a.x = x; a.ldx = ldx; a.rows = rows; a.cols = cols; a.w = weight; a.b = bias; a.eps = eps; a.y = y; a.ldy = ldy;
  a.mean = mean; a.rstd = rstd;
  a.x_codes = x_codes; a.x_exps = x_exps; a.y_codes = y_codes; a.y_exps = y_exps;
  return launched(gc::launch_layernorm_forward(dtype, wdtype, a, to_stream(stream)), "gc_layernorm_forward");
}

int gc_layernorm_backward_workspace(int64_t rows, int64_t cols, size_t* bytes) {
  GC_REQUIRE(bytes != nullptr, "bytes is NULL");
  *bytes = 0;
  GC_TRY(check_shape(GC_F32, rows, cols));
  *bytes = gc::layernorm_backward_workspace(rows, cols);
  return ok();
}

int gc_layernorm_backward(int dtype, const void* dy, int64_t lddy, const void* x, int64_t ldx, const int8_t* x_codes,
                          const uint8_t* x_exps, int64_t rows, int64_t cols, int wdtype, const void* weight,
                          const float* mean, const float* rstd, void* dx, int64_t lddx, float* dw, float* db,
                          int accumulate, void* workspace, size_t workspace_bytes, void* stream) {
  GC_TRY(check_shape(dtype, rows, cols));
  GC_TRY(check_weight_type(dtype, wdtype));
  GC_REQUIRE(f32_ok(dw) && f32_ok(db), "dw and db must be 4-byte aligned");
  gc::LnBwdArgs a{};
  a.rows = rows; a.cols = cols; a.dw = dw; a.db = db; a.accumulate = accumulate;
  if (rows == 0) {
    if (cols == 0 || accumulate || (!dw && !db)) return ok();
    return launched(gc::launch_layernorm_backward(dtype, wdtype, a, to_stream(stream)), "gc_layernorm_backward");
  }
  GC_REQUIRE(cols >= 1, "cols must be >= 1");
  GC_REQUIRE((x != nullptr) != (x_codes != nullptr), "exactly one of x and its checkpoint");
  GC_TRY(check_matrix("dy", dy, lddy, dtype, rows, cols));
  if (x) GC_TRY(check_matrix("x", x, ldx, dtype, rows, cols));
  else GC_TRY(check_ckpt("x", x_codes, x_exps, rows, cols));
  GC_REQUIRE(aligned(weight, (size_t)elem_size(wdtype)), "weight must be aligned to its element");
  GC_REQUIRE(mean && rstd && f32_ok(mean) && f32_ok(rstd), "mean and rstd must be non-NULL and 4-byte aligned");
  GC_TRY(check_matrix("dx", dx, lddx, dtype, rows, cols));
  const size_t need = gc::layernorm_backward_workspace(rows, cols);
  GC_TRY(check_workspace(workspace, workspace_bytes, need));
  GC_TRY(check_apart({use("dy", false, dy, lddy, dtype, rows, cols), use("dx", true, dx, lddx, dtype, rows, cols),
                      use("x", false, x, ldx, dtype, rows, cols),
                      use_bytes("codes", false, x_codes, codes_of(rows, cols)), use_bytes("exponents", false, x_exps, codes_of(rows, cols) / 32),
                      use("weight", false, weight, cols, wdtype, 1, cols), use_bytes("mean", false, mean, rows * 4),
                      use_bytes("rstd", false, rstd, rows * 4), use_bytes("dw", true, dw, cols * 4), use_bytes("db", true, db, cols * 4),
                      use_bytes("workspace", true, workspace, (int64_t)need)}));
  a.dy = dy; a.lddy = lddy; a.x = x; a.ldx = ldx; a.x_codes = x_codes; a.x_exps = x_exps; a.w = weight;
  a.mean = mean; a.rstd = rstd; a.dx = dx; a.lddx = lddx; a.ws = workspace;
  return launched(gc::launch_layernorm_backward(dtype, wdtype, a, to_stream(stream)), "gc_layernorm_backward");
}

static int check_linear(int dtype, int64_t rows, int64_t in_features, int64_t out_features) {
  GC_TRY(check_shape(dtype, rows, in_features));
  GC_REQUIRE(in_features >= 1 && in_features <= kMaxFeatures && out_features >= 1 && out_features <= kMaxFeatures,
             "in_features and out_features must lie in [1, 2^22]");
  return GC_OK;
}

int gc_linear_wgrad_workspace(int dtype, int64_t rows, int64_t in_features, int64_t out_features, size_t* bytes) {
  GC_REQUIRE(bytes != nullptr, "bytes is NULL");
  *bytes = 0;
  GC_TRY(check_linear(dtype, rows, in_features, out_features));
  *bytes = gc::wgrad_workspace(dtype, rows, in_features, out_features);
  return ok();
}

int gc_linear_wgrad(int dtype, const void* dy, int64_t lddy, const int8_t* codes, const uint8_t* exps, int64_t rows,
                    int64_t in_features, int64_t out_features, float* dw, int64_t lddw, float* db, int accumulate,
                    void* workspace, size_t workspace_bytes, void* stream) {
  GC_TRY(check_linear(dtype, rows, in_features, out_features));
  GC_TRY(check_matrix("dw", dw, lddw, GC_F32, out_features, in_features));
  GC_REQUIRE(f32_ok(db), "db must be 4-byte aligned");
  gc::WgradArgs a{};
  a.rows = rows; a.in = in_features; a.out = out_features; a.dw = dw; a.lddw = lddw; a.db = db; a.accumulate = accumulate;
  if (rows == 0) {
    if (accumulate) return ok();
    return launched(gc::launch_wgrad(dtype, a, to_stream(stream)), "gc_linear_wgrad");
  }
  GC_TRY(check_matrix("dy", dy, lddy, dtype, rows, out_features));
  GC_TRY(check_ckpt("the checkpoint's", codes, exps, rows, in_features));
  const size_t need = gc::wgrad_workspace(dtype, rows, in_features, out_features);
  GC_TRY(check_workspace(workspace, workspace_bytes, need));
  GC_TRY(check_apart({use("dy", false, dy, lddy, dtype, rows, out_features), use("dw", true, dw, lddw, GC_F32, out_features, in_features),
                      use_bytes("codes", false, codes, codes_of(rows, in_features)),
                      use_bytes("exponents", false, exps, codes_of(rows, in_features) / 32), use_bytes("db", true, db, out_features * 4),
                      use_bytes("workspace", true, workspace, (int64_t)need)}));
  a.dy = dy; a.lddy = lddy; a.codes = codes; a.exps = exps; a.ws = workspace;
  return launched(gc::launch_wgrad(dtype, a, to_stream(stream)), "gc_linear_wgrad");
}

}  // extern "C"
