// C-ABI entry points of the residual block's norms: argument checks and the
// kernels' arguments.  See include/moe.h for the contract of each call.
#include <math.h>
#include <string.h>

#include "moe_block.cuh"

namespace moe {
namespace {

bool is_float_type(int t) { return t == MOE_DTYPE_BF16 || t == MOE_DTYPE_FP32; }
size_t type_bytes(int t) { return t == MOE_DTYPE_FP32 ? 4 : 2; }

moe_status_t check_norm_desc(const moe_block_norm_desc_t* d) {
  if (!d) return MOE_ERR_NULL;
  if (d->T < 0 || d->T > kBlockMaxT || d->d < 1 || d->d > kBlockMaxD) return MOE_ERR_SHAPE;
  if (!is_float_type(d->dtype) || !is_float_type(d->res_dtype) || !is_float_type(d->param_dtype))
    return MOE_ERR_UNSUPPORTED;
  if (d->dtype == MOE_DTYPE_FP32 && d->res_dtype != MOE_DTYPE_FP32) return MOE_ERR_UNSUPPORTED;
  if (d->pre_norm < MOE_NORM_NONE || d->pre_norm > MOE_NORM_LAYER ||
      d->post_norm < MOE_NORM_NONE || d->post_norm > MOE_NORM_LAYER ||
      d->gate < MOE_GATE_NONE || d->gate > MOE_GATE_FULL || d->gate_act < MOE_GATE_ACT_NONE ||
      d->gate_act > MOE_GATE_ACT_TANH)
    return MOE_ERR_UNSUPPORTED;
  if (!(d->pre_eps > 0.0f) || !(d->post_eps > 0.0f) || !isfinite(d->pre_eps) ||
      !isfinite(d->post_eps) || !isfinite(d->pre_offset) || !isfinite(d->post_offset) ||
      !isfinite(d->res_scale) || !isfinite(d->branch_scale))
    return MOE_ERR_SHAPE;
  return MOE_OK;
}

// Collects a call's pointers: their status, and whether all can be moved 16
// bytes at a time.
struct Checker {
  const moe_block_norm_desc_t* d;
  moe_status_t st = MOE_OK;
  bool vec;
  explicit Checker(const moe_block_norm_desc_t* desc) : d(desc), vec(desc->d % kUnit == 0) {}

  void fail(moe_status_t s) {
    if (st == MOE_OK) st = s;
  }
  BlockRows rows(const moe_rows_t& r, int type, bool required, long long n_rows) {
    if (!r.p) {
      if (required) fail(MOE_ERR_NULL);
      return {nullptr, 0, 0};
    }
    const size_t b = type_bytes(type);
    const uintptr_t at = reinterpret_cast<uintptr_t>(r.p);
    if (at % b || r.ld < 0 || (n_rows > 1 && r.ld < d->d)) fail(MOE_ERR_SHAPE);
    const size_t whole = kUnit * b;   // a unit: 16 or 32 bytes
    if (at % whole || (n_rows > 1 && (static_cast<size_t>(r.ld) * b) % whole)) vec = false;
    const size_t step = n_rows > 1 ? static_cast<size_t>(r.ld) * b / 16 : 0;
    if (step > UINT32_MAX) vec = false;
    return {static_cast<char*>(r.p), static_cast<long long>(r.ld), static_cast<uint32_t>(step)};
  }
  BlockRows rows(const moe_rows_t& r, int type, bool required) {
    return rows(r, type, required, d->T);
  }
  // a parameter vector or its gradient
  void* vector(const void* v) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(v);
    if (at % type_bytes(d->param_dtype)) fail(MOE_ERR_SHAPE);
    if (at % 16) vec = false;
    return const_cast<void*>(v);
  }
  BlockNorm norm(bool pre, const void* w, const void* b) {
    BlockNorm n;
    n.kind = pre ? d->pre_norm : d->post_norm;
    n.eps = pre ? d->pre_eps : d->post_eps;
    n.off = pre ? d->pre_offset : d->post_offset;
    n.w = n.kind == MOE_NORM_NONE ? nullptr : vector(w);
    n.b = n.kind == MOE_NORM_NONE ? nullptr : vector(b);
    return n;
  }
  // (without tokens a token or full gate has no values and may be absent)
  BlockRows gate(const moe_rows_t& r) {
    if (d->gate == MOE_GATE_NONE) return {nullptr, 0, 0};
    if (d->gate == MOE_GATE_FULL) return rows(r, d->dtype, d->T > 0);
    if (!r.p && (d->gate == MOE_GATE_CHANNEL || d->T > 0)) {
      fail(MOE_ERR_NULL);
      return {nullptr, 0, 0};
    }
    if (d->gate == MOE_GATE_CHANNEL) return {static_cast<char*>(vector(r.p)), 0, 0};
    return token(r);
  }
  BlockRows token(const moe_rows_t& r) {
    if (r.p && (reinterpret_cast<uintptr_t>(r.p) % 4 || r.ld < 0 || (d->T > 1 && r.ld < 1)))
      fail(MOE_ERR_SHAPE);
    return {static_cast<char*>(r.p), static_cast<long long>(r.ld), 0};
  }
};

// (the gate is the post norm's: a pre norm's call has no gate to read)
void fill(BlockArgs& a, const moe_block_norm_desc_t* d, bool vec, bool post) {
  a.T = d->T;
  a.d = d->d;
  a.vec = vec;
  a.p32 = d->param_dtype == MOE_DTYPE_FP32;
  a.gate = post ? d->gate : MOE_GATE_NONE;
  a.gate_act = post ? d->gate_act : MOE_GATE_ACT_NONE;
  a.res_scale = d->res_scale;
  a.branch_scale = d->branch_scale;
}

size_t bwd_ws_bytes(const moe_block_norm_desc_t* d) {
  const size_t parts = d->T < kBlockBwdMaxParts ? d->T : kBlockBwdMaxParts;
  return parts * 4 * d->d * sizeof(float) + 256;
}

cudaError_t launch_fwd(const moe_block_norm_desc_t* d, const BlockArgs& a, bool post, int sms,
                       cudaStream_t s) {
  if (d->dtype == MOE_DTYPE_FP32) return launch_block_fwd_types<float, float>(a, post, sms, s);
  if (d->res_dtype == MOE_DTYPE_FP32)
    return launch_block_fwd_types<__nv_bfloat16, float>(a, post, sms, s);
  return launch_block_fwd_types<__nv_bfloat16, __nv_bfloat16>(a, post, sms, s);
}

moe_status_t to_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

moe_status_t run_bwd(const moe_block_norm_desc_t* desc, Checker& c, BlockArgs& a, BlockGrads& o,
                     void* ws, size_t ws_bytes, cudaStream_t stream) {
  if (!ws) c.fail(MOE_ERR_NULL);
  if (reinterpret_cast<uintptr_t>(ws) % 16) c.fail(MOE_ERR_SHAPE);
  if (c.st != MOE_OK) return c.st;
  if (ws_bytes < bwd_ws_bytes(desc)) return MOE_ERR_WORKSPACE;
  int sms;
  const moe_status_t st = current_device(&sms, &a.status);
  if (st != MOE_OK) return st;
  fill(a, desc, c.vec, o.post);
  a.part = static_cast<float*>(ws);
  return to_status(launch_block_bwd(a, o, desc->dtype, desc->res_dtype, sms, stream));
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_block_norm_workspace_size(const moe_block_norm_desc_t* desc, size_t* bytes) {
  if (!bytes) return MOE_ERR_NULL;
  const moe_status_t st = check_norm_desc(desc);
  if (st != MOE_OK) return st;
  *bytes = bwd_ws_bytes(desc);
  return MOE_OK;
}

moe_status_t moe_block_pre_norm_fwd(const moe_block_norm_desc_t* desc, moe_rows_t res,
                                    const void* w, const void* b, moe_rows_t x,
                                    cudaStream_t stream) {
  moe_status_t st = check_norm_desc(desc);
  if (st != MOE_OK) return st;
  if (desc->pre_norm == MOE_NORM_NONE) return MOE_ERR_UNSUPPORTED;
  if (desc->T == 0) return MOE_OK;
  BlockArgs a;
  memset(&a, 0, sizeof(a));
  Checker c(desc);
  a.res = c.rows(res, desc->res_dtype, true);
  a.x = c.rows(x, desc->dtype, true);
  a.pre = c.norm(true, w, b);
  if (c.st != MOE_OK) return c.st;
  int sms;
  if ((st = current_device(&sms, &a.status)) != MOE_OK) return st;
  fill(a, desc, c.vec, false);
  return to_status(launch_fwd(desc, a, false, sms, stream));
}

moe_status_t moe_block_post_norm_fwd(const moe_block_norm_desc_t* desc, moe_rows_t res,
                                     moe_rows_t y, const moe_block_params_t* params,
                                     moe_rows_t res_out, moe_rows_t x,
                                     const moe_routed_rows_t* routed, cudaStream_t stream) {
  moe_status_t st = check_norm_desc(desc);
  if (st != MOE_OK) return st;
  if (!params) return MOE_ERR_NULL;
  if (x.p && desc->pre_norm == MOE_NORM_NONE) return MOE_ERR_UNSUPPORTED;
  if (routed && (routed->k < 1 || routed->k > kMaxTopK || routed->capacity < 0))
    return MOE_ERR_SHAPE;
  if (desc->T == 0) return MOE_OK;
  BlockArgs a;
  memset(&a, 0, sizeof(a));
  Checker c(desc);
  a.res = c.rows(res, desc->res_dtype, true);
  a.res_out = c.rows(res_out, desc->res_dtype, true);
  a.x = c.rows(x, desc->dtype, false);
  a.y = c.rows(y, desc->dtype, true, routed ? routed->capacity : desc->T);
  a.post = c.norm(false, params->post_w, params->post_b);
  if (a.x.p) a.pre = c.norm(true, params->pre_w, params->pre_b);
  a.gate_rows = c.gate(params->gate);
  if (routed) {
    if (!routed->row_of || !routed->topk_w) c.fail(MOE_ERR_NULL);
    if ((reinterpret_cast<uintptr_t>(routed->row_of) | reinterpret_cast<uintptr_t>(routed->topk_w)) % 4)
      c.fail(MOE_ERR_SHAPE);
    a.row_of = routed->row_of;
    a.topk_w = routed->topk_w;
    a.k = routed->k;
    a.capacity = routed->capacity;
    a.y_out = c.rows(routed->y_out, desc->dtype, false);
  }
  if (c.st != MOE_OK) return c.st;
  int sms;
  if ((st = current_device(&sms, &a.status)) != MOE_OK) return st;
  fill(a, desc, c.vec, true);
  return to_status(launch_fwd(desc, a, true, sms, stream));
}

moe_status_t moe_block_pre_norm_bwd(const moe_block_norm_desc_t* desc, moe_rows_t dx,
                                    moe_rows_t res, const void* w, moe_rows_t dres_in,
                                    float dres_scale, moe_rows_t dres, void* dw, void* db,
                                    void* ws, size_t ws_bytes, cudaStream_t stream) {
  const moe_status_t st = check_norm_desc(desc);
  if (st != MOE_OK) return st;
  if (desc->pre_norm == MOE_NORM_NONE) return MOE_ERR_UNSUPPORTED;
  if (!isfinite(dres_scale)) return MOE_ERR_SHAPE;
  const bool rows = desc->T > 0;
  BlockArgs a;
  memset(&a, 0, sizeof(a));
  BlockGrads o;
  memset(&o, 0, sizeof(o));
  Checker c(desc);
  a.dx = c.rows(dx, desc->dtype, rows);
  a.res = c.rows(res, desc->res_dtype, rows);
  a.dres_in = c.rows(dres_in, desc->res_dtype, false);
  a.dres = c.rows(dres, desc->res_dtype, rows);
  a.pre = c.norm(true, w, nullptr);
  a.dres_scale = dres_scale;
  o.pre = true;
  o.dpre_w = c.vector(dw);
  o.dpre_b = c.vector(db);
  o.bias = db != nullptr;
  return run_bwd(desc, c, a, o, ws, ws_bytes, stream);
}

moe_status_t moe_block_post_norm_bwd(const moe_block_norm_desc_t* desc, moe_rows_t dres_in,
                                     float dres_scale, moe_rows_t dx, moe_rows_t res_out,
                                     moe_rows_t y, const moe_block_params_t* params,
                                     moe_rows_t dres, moe_rows_t dy,
                                     const moe_block_params_t* grads, void* ws, size_t ws_bytes,
                                     cudaStream_t stream) {
  const moe_status_t st = check_norm_desc(desc);
  if (st != MOE_OK) return st;
  if (!params || !grads) return MOE_ERR_NULL;
  if (!isfinite(dres_scale)) return MOE_ERR_SHAPE;
  const bool rows = desc->T > 0;
  if (dx.p && desc->pre_norm == MOE_NORM_NONE) return MOE_ERR_UNSUPPORTED;
  if (rows && !dx.p && !dres_in.p) return MOE_ERR_NULL;
  BlockArgs a;
  memset(&a, 0, sizeof(a));
  BlockGrads o;
  memset(&o, 0, sizeof(o));
  Checker c(desc);
  a.dres_in = c.rows(dres_in, desc->res_dtype, false);
  a.dx = c.rows(dx, desc->dtype, false);
  a.y = c.rows(y, desc->dtype, rows);
  a.dres = c.rows(dres, desc->res_dtype, false);
  a.dy = c.rows(dy, desc->dtype, rows);
  a.post = c.norm(false, params->post_w, params->post_b);
  a.gate_rows = c.gate(params->gate);
  a.dres_scale = dres_scale;
  o.post = true;
  // without rows the next norm's gradients are still wanted as zeros
  o.pre = dx.p != nullptr || (!rows && (grads->pre_w || grads->pre_b));
  if (o.pre) {
    a.res = c.rows(res_out, desc->res_dtype, rows);
    a.pre = c.norm(true, params->pre_w, nullptr);
    o.dpre_w = c.vector(grads->pre_w);
    o.dpre_b = c.vector(grads->pre_b);
  }
  if (desc->post_norm != MOE_NORM_NONE) {
    o.dpost_w = c.vector(grads->post_w);
    o.dpost_b = c.vector(grads->post_b);
  }
  if (grads->gate.p) {
    if (desc->gate == MOE_GATE_CHANNEL) o.dgate = c.vector(grads->gate.p);
    if (desc->gate == MOE_GATE_TOKEN) a.dgate = c.token(grads->gate);
    if (desc->gate == MOE_GATE_FULL) a.dgate = c.rows(grads->gate, desc->dtype, false);
  }
  o.bias = o.dpre_b || o.dpost_b || (o.dgate && a.post.b);
  return run_bwd(desc, c, a, o, ws, ws_bytes, stream);
}

}  // extern "C"
