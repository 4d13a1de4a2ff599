// C ABI of the operators around the MoE layer: the free products (per expert
// and dense), the activation backward and residual dropout. Argument checks
// and launches; include/moe.h documents every argument.
#include <cmath>

#include "moe_common.cuh"

#include "moe_internal.h"

namespace moe {
namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int rc_of(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

// A copy of the configuration with every stride filled in.
struct Product {
  moe_gemm_config c;
  int rc;
};

// Which operands a call has: their strides are checked, the others' ignored.
struct Uses {
  bool x, w, y;
  int64_t r_width, z_width;  // widths of residual and z rows, 0 if the call has none
};

constexpr int64_t kFar = 1LL << 36;  // elements: tensor maps hold strides of less than 2^40 bytes

bool stride_ok(int64_t ld, int64_t width, bool bf16, int& rc) {
  if (ld < width) rc = MOE_ERR_INVALID_ARG;
  else if (ld > kFar || (bf16 && ld % 8 != 0)) rc = MOE_ERR_UNSUPPORTED;
  return rc == MOE_OK;
}

Product check(const moe_gemm_config* cfg, bool dense, const Uses& u) {
  Product p{};
  p.rc = MOE_ERR_INVALID_ARG;
  if (cfg == nullptr) return p;
  moe_gemm_config& c = p.c = *cfg;
  if (c.rows < 0 || c.n <= 0 || c.k <= 0 || c.groups <= 0) return p;
  if (c.dtype != MOE_DTYPE_BF16 && c.dtype != MOE_DTYPE_F32) return p;
  if (c.act < MOE_ACT_NONE || c.act > MOE_ACT_SILU) return p;
  if (dense && c.groups != 1) return p;
  p.rc = MOE_ERR_UNSUPPORTED;
  // row and column indices stay below 2^31, a tile past the last one included
  constexpr int32_t kMost = INT32_MAX - 1024;
  // and bf16 widths at most what the tensor-core tiles' bounded waits are known to last for
  constexpr int32_t kMostBf16 = 1 << 26;
  const int32_t most = c.dtype == MOE_DTYPE_BF16 ? kMostBf16 : kMost;
  if (c.rows > kMost || c.n > most || c.k > most) return p;
  if (c.groups > MOE_MAX_E || static_cast<int64_t>(c.groups) * c.n >= (1LL << 31)) return p;
  if (c.ldx == 0) c.ldx = c.k;
  if (c.ldw == 0) c.ldw = c.k;
  if (c.ldy == 0) c.ldy = c.n;
  if (c.ldr == 0) c.ldr = u.r_width;
  if (c.ldz == 0) c.ldz = u.z_width;
  const bool bf16 = c.dtype == MOE_DTYPE_BF16;
  p.rc = MOE_OK;
  if (u.x && !stride_ok(c.ldx, c.k, bf16, p.rc)) return p;
  if (u.y && !stride_ok(c.ldy, c.n, bf16, p.rc)) return p;
  if (u.r_width && !stride_ok(c.ldr, u.r_width, bf16, p.rc)) return p;
  if (u.z_width && !stride_ok(c.ldz, u.z_width, bf16, p.rc)) return p;
  if (u.w) {
    if (!stride_ok(c.ldw, c.k, bf16, p.rc)) return p;
    if (c.groups == 1) {
      c.w_stride = c.ldw;  // leads nowhere
    } else if (c.n - 1 > kFar / c.ldw) {  // no group stride is long enough
      p.rc = MOE_ERR_UNSUPPORTED;
    } else {
      if (c.w_stride == 0) c.w_stride = c.ldw * c.n;
      stride_ok(c.w_stride, (c.n - 1) * c.ldw + c.k, bf16, p.rc);
    }
  }
  return p;
}

MatmulPlan plan_product(int dtype, MatmulMode mode, const MatmulArgs& a, int sms) {
  const bool f32 = dtype == MOE_DTYPE_F32;
  if (mode == MatmulMode::kForward && (f32 ? matmul_few_rows_f32(a) : matmul_few_rows(a, sms)))
    return {Form::kFewRows, 0, 1, 0};
  return f32 ? plan_matmul_f32(mode, a, sms) : plan_matmul_tc(mode, a, sms);
}

// Products of 2^31 tiles or more leave the bf16 tiles' 32-bit indices.
bool too_many(int dtype, const MatmulPlan& plan) { return dtype == MOE_DTYPE_BF16 && plan.tiles >= 1LL << 31; }

int launch_product(int dtype, MatmulMode mode, const MatmulArgs& a, cudaStream_t s) {
  const bool f32 = dtype == MOE_DTYPE_F32;
  const int sms = device_sm_count();
  const MatmulPlan plan = plan_product(dtype, mode, a, sms);
  if (too_many(dtype, plan)) return MOE_ERR_UNSUPPORTED;
  if (plan.form == Form::kFewRows) return rc_of(f32 ? launch_matmul_rows_f32(a, s) : launch_matmul_rows(a, sms, s));
  return rc_of(f32 ? launch_matmul_f32(mode, plan, a, sms, s) : launch_matmul_tc(mode, plan, a, sms, s));
}

int forward(const moe_gemm_config* cfg, bool dense, const void* x, const int32_t* offsets, const void* w,
            const float* bias, const void* residual, void* preact, void* y, int32_t* status, cudaStream_t s) {
  const Product p =
      check(cfg, dense, {true, true, true, residual && cfg ? cfg->n : 0, preact && cfg ? cfg->n : 0});
  if (p.rc != MOE_OK) return p.rc;
  const moe_gemm_config& c = p.c;
  if (!w || (!dense && !offsets) || (c.rows > 0 && (!x || !y))) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(y, 16) || !aligned(residual, 16) || !aligned(preact, 16) ||
      !aligned(bias, 4) || !aligned(offsets, 4) || !aligned(status, 4))
    return MOE_ERR_UNSUPPORTED;
  if (c.rows == 0) return MOE_OK;
  MatmulArgs a{};
  a.a = x, a.b = w, a.offsets = offsets, a.groups = c.groups, a.rows = c.rows;
  a.n = c.n, a.k = c.k, a.lda = c.ldx, a.ldb = c.ldw, a.b_stride = c.w_stride, a.ldd = c.ldy;
  a.bias = bias, a.preact = preact, a.residual = residual, a.ldz = c.ldz, a.ldr = c.ldr;
  a.d = y, a.act = c.act, a.status = status;
  a.vec = c.k % 4 == 0 && c.ldx % 4 == 0 && c.ldw % 4 == 0 && c.w_stride % 4 == 0;
  a.vec_out = c.ldy % 4 == 0 && (!residual || c.ldr % 4 == 0) && (!preact || c.ldz % 4 == 0);
  return launch_product(c.dtype, MatmulMode::kForward, a, s);
}

int dgrad(const moe_gemm_config* cfg, bool dense, const void* dy, const int32_t* offsets, const void* w, const void* z,
          const void* residual, void* dx, int32_t* status, cudaStream_t s) {
  const Product p = check(cfg, dense, {true, true, true, residual && cfg ? cfg->k : 0, z && cfg ? cfg->k : 0});
  if (p.rc != MOE_OK) return p.rc;
  const moe_gemm_config& c = p.c;
  if (!w || (!dense && !offsets) || (c.rows > 0 && (!dy || !dx))) return MOE_ERR_INVALID_ARG;
  if (!aligned(dy, 16) || !aligned(w, 16) || !aligned(z, 16) || !aligned(residual, 16) || !aligned(dx, 16) ||
      !aligned(offsets, 4) || !aligned(status, 4))
    return MOE_ERR_UNSUPPORTED;
  if (c.rows == 0) return MOE_OK;
  MatmulArgs a{};
  a.a = dy, a.b = w, a.offsets = offsets, a.groups = c.groups, a.rows = c.rows;
  a.n = c.k, a.k = c.n, a.lda = c.ldy, a.ldb = c.ldw, a.b_stride = c.w_stride, a.ldd = c.ldx;
  a.z = z, a.residual = residual, a.ldz = c.ldz, a.ldr = c.ldr;
  a.d = dx, a.act = c.act, a.status = status;
  a.vec = c.n % 4 == 0 && c.k % 4 == 0 && c.ldy % 4 == 0 && c.ldw % 4 == 0 && c.w_stride % 4 == 0;
  a.vec_out = c.ldx % 4 == 0 && (!residual || c.ldr % 4 == 0) && (!z || c.ldz % 4 == 0);
  return launch_product(c.dtype, MatmulMode::kDgrad, a, s);
}

int wgrad(const moe_gemm_config* cfg, bool dense, const void* dy, const int32_t* offsets, const void* x, float* dw,
          float* dbias, int32_t* status, cudaStream_t s) {
  const Product p = check(cfg, dense, {true, false, true, 0, 0});
  if (p.rc != MOE_OK) return p.rc;
  const moe_gemm_config& c = p.c;
  if ((!dense && !offsets) || (c.rows > 0 && (!dy || !x))) return MOE_ERR_INVALID_ARG;
  if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(dw, 4) || !aligned(dbias, 4) || !aligned(offsets, 4) ||
      !aligned(status, 4))
    return MOE_ERR_UNSUPPORTED;
  // no rows at all: the gradients are zero (every group is empty whatever the offsets hold)
  if (c.rows == 0) {
    const size_t each = static_cast<size_t>(c.groups) * c.n;
    cudaError_t e = dw ? cudaMemsetAsync(dw, 0, each * c.k * 4, s) : cudaSuccess;
    if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, each * 4, s);
    return rc_of(e);
  }
  if (dw) {
    MatmulArgs a{};
    a.a = dy, a.b = x, a.offsets = offsets, a.groups = c.groups, a.rows = c.rows;
    a.m = c.n, a.n = c.k, a.lda = c.ldy, a.ldb = c.ldx, a.ldd = c.k;
    a.d = dw, a.status = status;
    a.vec = c.n % 4 == 0 && c.k % 4 == 0 && c.ldy % 4 == 0 && c.ldx % 4 == 0;
    a.vec_out = c.k % 4 == 0 && aligned(dw, 16);
    const int rc = launch_product(c.dtype, MatmulMode::kWgrad, a, s);
    if (rc != MOE_OK) return rc;
  }
  if (dbias)
    return rc_of(launch_column_sums(c.dtype, dy, c.ldy, offsets, c.groups, c.rows, c.n, dbias, dw ? nullptr : status,
                                    c.n % 4 == 0 && c.ldy % 4 == 0, s));
  return MOE_OK;
}

// The dropout arguments in their kernel form; false if p or rng is no good.
bool dropout_args(double p, const uint64_t* rng, uint64_t offset, DropoutArgs* d) {
  if (!(p >= 0.0 && p < 1.0) || (p > 0.0 && rng == nullptr)) return false;
  d->rng = reinterpret_cast<const unsigned long long*>(rng);
  d->offset = offset;
  d->cut = static_cast<uint32_t>(std::floor(p * 4294967296.0));
  d->scale = static_cast<float>(1.0 / (1.0 - p));
  return true;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int32_t moe_grouped_gemm(const moe_gemm_config* cfg, const void* x, const int32_t* offsets, const void* w,
                         const float* bias, const void* residual, void* preact, void* y, int32_t* status_dev,
                         moe_stream_t stream) {
  return forward(cfg, false, x, offsets, w, bias, residual, preact, y, status_dev, static_cast<cudaStream_t>(stream));
}

int32_t moe_grouped_gemm_dgrad(const moe_gemm_config* cfg, const void* dy, const int32_t* offsets, const void* w,
                               const void* z, const void* residual, void* dx, int32_t* status_dev,
                               moe_stream_t stream) {
  return dgrad(cfg, false, dy, offsets, w, z, residual, dx, status_dev, static_cast<cudaStream_t>(stream));
}

int32_t moe_grouped_gemm_wgrad(const moe_gemm_config* cfg, const void* dy, const int32_t* offsets, const void* x,
                               float* dw, float* dbias, int32_t* status_dev, moe_stream_t stream) {
  return wgrad(cfg, false, dy, offsets, x, dw, dbias, status_dev, static_cast<cudaStream_t>(stream));
}

int32_t moe_linear(const moe_gemm_config* cfg, const void* x, const void* w, const float* bias, const void* residual,
                   void* preact, void* y, int32_t* status_dev, moe_stream_t stream) {
  return forward(cfg, true, x, nullptr, w, bias, residual, preact, y, status_dev, static_cast<cudaStream_t>(stream));
}

int32_t moe_linear_dgrad(const moe_gemm_config* cfg, const void* dy, const void* w, const void* z,
                         const void* residual, void* dx, int32_t* status_dev, moe_stream_t stream) {
  return dgrad(cfg, true, dy, nullptr, w, z, residual, dx, status_dev, static_cast<cudaStream_t>(stream));
}

int32_t moe_linear_wgrad(const moe_gemm_config* cfg, const void* dy, const void* x, float* dw, float* dbias,
                         int32_t* status_dev, moe_stream_t stream) {
  return wgrad(cfg, true, dy, nullptr, x, dw, dbias, status_dev, static_cast<cudaStream_t>(stream));
}

int32_t moe_product_form_used(const moe_gemm_config* cfg, int32_t product, int32_t sms, int32_t* form) {
  if (form == nullptr || sms <= 0 || product < MOE_PRODUCT_FORWARD || product > MOE_PRODUCT_WGRAD)
    return MOE_ERR_INVALID_ARG;
  const bool weight = product == MOE_PRODUCT_WGRAD;
  const Product p = check(cfg, false, {true, !weight, true, 0, 0});
  if (p.rc != MOE_OK) return p.rc;
  const moe_gemm_config& c = p.c;
  MatmulArgs a{};
  a.groups = c.groups, a.rows = c.rows, a.m = c.n;
  a.n = product == MOE_PRODUCT_FORWARD ? c.n : c.k, a.k = product == MOE_PRODUCT_FORWARD ? c.k : c.n;
  const MatmulMode mode = product == MOE_PRODUCT_FORWARD ? MatmulMode::kForward
                          : weight                       ? MatmulMode::kWgrad
                                                         : MatmulMode::kDgrad;
  const MatmulPlan plan = plan_product(c.dtype, mode, a, sms);
  if (too_many(c.dtype, plan)) return MOE_ERR_UNSUPPORTED;
  form[0] = plan.form == Form::kFewRows  ? MOE_FORM_FEW_ROWS
            : plan.form == Form::kSingle ? MOE_FORM_SINGLE
            : plan.form == Form::kPair   ? MOE_FORM_PAIR
                                         : MOE_FORM_SPLIT;
  form[1] = plan.bn;
  form[2] = plan.split;
  return MOE_OK;
}

int32_t moe_act_backward(const moe_gemm_config* cfg, const void* dy, const void* z, void* dz, moe_stream_t stream) {
  if (cfg == nullptr) return MOE_ERR_INVALID_ARG;
  moe_gemm_config matrix = *cfg;
  matrix.k = matrix.groups = 1;  // no product: neither counts
  const Product p = check(&matrix, true, {false, false, true, cfg->n, cfg->n});
  if (p.rc != MOE_OK) return p.rc;
  const moe_gemm_config& c = p.c;
  if (c.rows > 0 && (!dy || !z || !dz)) return MOE_ERR_INVALID_ARG;
  if (!aligned(dy, 16) || !aligned(z, 16) || !aligned(dz, 16)) return MOE_ERR_UNSUPPORTED;
  if (c.rows == 0) return MOE_OK;
  const bool vec = c.n % 4 == 0 && c.ldy % 4 == 0 && c.ldz % 4 == 0 && c.ldr % 4 == 0;
  return rc_of(launch_act_backward(c.dtype, dy, c.ldy, z, c.ldz, dz, c.ldr, c.rows, c.n, c.act, vec,
                                   static_cast<cudaStream_t>(stream)));
}

int32_t moe_dropout(int32_t rows, int32_t cols, int32_t dtype, const void* x, int64_t ldx, const void* residual,
                    int64_t ldr, void* y, int64_t ldy, double p, const uint64_t* rng, uint64_t offset,
                    moe_stream_t stream) {
  DropoutArgs d{};
  if (rows < 0 || cols <= 0 || (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F32)) return MOE_ERR_INVALID_ARG;
  if (!dropout_args(p, rng, offset, &d)) return MOE_ERR_INVALID_ARG;
  if (rows > 0 && (!x || !y)) return MOE_ERR_INVALID_ARG;
  if (ldx == 0) ldx = cols;
  if (ldr == 0 || !residual) ldr = cols;
  if (ldy == 0) ldy = cols;
  if (ldx < cols || ldr < cols || ldy < cols) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(y, 16) || !aligned(rng, 8)) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  return rc_of(launch_dropout(dtype, rows, cols, x, ldx, residual, ldr, y, ldy, d, static_cast<cudaStream_t>(stream)));
}

int32_t moe_unpermute_combine_dropout(const moe_config* cfg, const void* y_perm, const int32_t* dest_row,
                                      const float* topk_gate, const void* residual, double p, const uint64_t* rng,
                                      uint64_t offset, void* y, moe_stream_t stream) {
  int32_t tiles;
  const int rc = moe_gemm_tiles_used(cfg, &tiles);  // the layer's configuration check
  if (rc != MOE_OK) return rc;
  DropoutArgs d{};
  if (!dropout_args(p, rng, offset, &d)) return MOE_ERR_INVALID_ARG;
  if (cfg->T > 0 && (!y_perm || !dest_row || !topk_gate || !y)) return MOE_ERR_INVALID_ARG;
  if (!aligned(y_perm, 16) || !aligned(y, 16) || !aligned(residual, 16) || !aligned(dest_row, 4) ||
      !aligned(topk_gate, 4) || !aligned(rng, 8))
    return MOE_ERR_UNSUPPORTED;
  const int64_t rows = cfg->layout == MOE_LAYOUT_PADDED ? static_cast<int64_t>(cfg->E) * cfg->capacity
                                                         : static_cast<int64_t>(cfg->T) * cfg->k;
  return rc_of(launch_combine_dropout(cfg->dtype, y_perm, static_cast<int>(rows), dest_row, topk_gate, residual, d, y,
                                      cfg->T, cfg->k, cfg->d, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
