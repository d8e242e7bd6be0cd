// C ABI of the layer operators: argument checks, workspace and the choice of
// kernels.
#include <algorithm>
#include <cmath>

#include "oz2_entry.cuh"
#include "oz2_layers.cuh"

namespace oz2 {
namespace {

bool is_16bit(int t) { return t == OZ2_BF16 || t == OZ2_F16; }
bool dropout_ok(double p) { return p >= 0.0 && p <= 1.0; }  // false for NaN

Dropout make_dropout(double p, uint64_t seed, uint64_t offset) {
  Dropout d;
  d.threshold = static_cast<uint32_t>(std::lround(65536.0 * p));
  d.limit = static_cast<uint32_t>((static_cast<uint64_t>(d.threshold) << 16) - 1);
  d.scale = d.threshold == 65536 ? 0.0f : 65536.0f / static_cast<float>(65536 - d.threshold);
  d.seed0 = static_cast<uint32_t>(seed);
  d.seed1 = static_cast<uint32_t>(seed >> 32);
  d.offset0 = static_cast<uint32_t>(offset);
  d.offset1 = static_cast<uint32_t>(offset >> 32);
  return d;
}

// Regions of the workspace, on 256-byte boundaries: sizes are collected first, addresses given out afterwards.
struct Carver {
  size_t used = 0;
  size_t take(size_t bytes) {
    const size_t at = used;
    used += (bytes + 255) / 256 * 256;
    return at;
  }
};

// A 16-bit matrix on its way into a product.  Rows that do not start on 16-byte
// boundaries are copied into the workspace first: one more read and write of
// the operand, for which the product itself has one fast form only.
struct Input {
  const void* p;
  int64_t rows, cols, ld;
  bool copy;
  size_t at;

  Input(const void* p_, int64_t rows_, int64_t cols_, int64_t ld_, bool used, Carver& c)
      : p(p_), rows(rows_), cols(cols_), ld(rows_ > 1 ? ld_ : ceil_div(cols_, 8) * 8), copy(false), at(0) {
    copy = used && rows > 0 && cols > 0 && !groups_aligned(p, ld, OZ2_BF16);
    if (copy) {
      ld = ceil_div(cols, 8) * 8;
      at = c.take(static_cast<size_t>(rows) * ld * 2);
    }
  }
  // The copy that is to be made, if any (from_ld: the leading dimension before it).
  PackJob place(uint8_t* base, int64_t from_ld) {
    if (!copy) return PackJob{};
    const void* from = p;
    p = base + at;
    return PackJob{rows, cols, from, from_ld, base + at, ld};
  }
};

oz2_status linear(const oz2_linear_args& a, cudaStream_t st) {
  if (a.m == 0 || a.n == 0) return OZ2_OK;
  const oz2_dtype dtype = static_cast<oz2_dtype>(a.dtype);
  DeviceResources res;
  oz2_status e = acquire_resources(st, 0, &res);
  if (e != OZ2_OK) return e;
  Epilogue ep{};
  ep.bias = a.bias;
  ep.residual = a.residual;
  ep.y = a.y;
  ep.z = a.preact;
  ep.ldr = a.ldr;
  ep.ldy = a.ldy;
  ep.ldz = a.ldz;
  ep.rows = a.m;
  ep.cols = a.n;
  ep.act = a.act;
  ep.scale = 1.0f;
  ep.drop = make_dropout(a.dropout, a.seed, a.offset);
  ep.vec = groups_aligned(a.y, a.ldy, dtype) && (!a.bias || groups_aligned(a.bias, 0, dtype)) &&
           (!a.residual || groups_aligned(a.residual, a.ldr, dtype)) && (!a.preact || groups_aligned(a.preact, a.ldz, dtype));
  Carver c;
  Input xi(a.x, a.m, a.k, a.ldx, true, c), wi(a.w, a.n, a.k, a.ldw, true, c);
  const LinearPlan plan(Operand{xi.p, xi.ld, false}, a.k, ep, res.num_sms);
  const size_t partial = c.take(plan.partial_bytes);
  e = acquire_resources(st, c.used, &res);
  if (e != OZ2_OK) return e;
  const PackJob x_job = xi.place(res.workspace, a.ldx), w_job = wi.place(res.workspace, a.ldw);
  OZ2_TRY(launch_pack(x_job, w_job, st));
  OZ2_TRY(launch_linear(plan, Operand{xi.p, xi.ld, false}, Operand{wi.p, wi.ld, false}, a.k, ep, dtype, res,
                        reinterpret_cast<float*>(res.workspace + partial), st));
  return OZ2_OK;
}

// A plain product, times scale, into out (no bias, activation, dropout or residual).
Epilogue plain_epilogue(void* out, int64_t ld, int64_t rows, int64_t cols, float scale, oz2_dtype dtype) {
  Epilogue ep{};
  ep.y = out;
  ep.scale = scale;
  ep.ldy = ld;
  ep.rows = rows;
  ep.cols = cols;
  ep.vec = groups_aligned(out, ld, dtype);
  return ep;
}

oz2_status linear_backward(const oz2_linear_backward_args& a, cudaStream_t st) {
  const int64_t m = a.m, k = a.k, n = a.n;
  const oz2_dtype dtype = static_cast<oz2_dtype>(a.dtype);
  void *dx = a.dx, *dw = a.dw, *dbias = a.dbias;
  const Dropout drop = make_dropout(a.dropout, a.seed, a.offset);
  DeviceResources res;
  oz2_status e = acquire_resources(st, 0, &res);
  if (e != OZ2_OK) return e;
  // sums over nothing
  if (m == 0 || n == 0) {
    if (dx && m > 0 && k > 0) OZ2_TRY(cudaMemset2DAsync(dx, a.lddx * 2, 0, k * 2, m, st));
    if (dw && n > 0 && k > 0) OZ2_TRY(cudaMemset2DAsync(dw, a.lddw * 2, 0, k * 2, n, st));
    if (dbias && n > 0) OZ2_TRY(cudaMemsetAsync(dbias, 0, n * 2, st));
    return OZ2_OK;
  }
  if (k == 0) dx = dw = nullptr;
  // dz is dy itself where nothing follows the product and its rows are aligned
  const bool products = dx || dw;
  const bool make_dz = products && (a.act != OZ2_ACT_NONE || drop.threshold != 0 || !groups_aligned(a.dy, a.lddy, dtype));
  const int64_t ld = make_dz ? ceil_div(n, 8) * 8 : a.lddy;
  Carver c;
  const size_t dz_at = c.take(make_dz ? static_cast<size_t>(m) * ld * 2 : 0);
  const int64_t sum_rows = dz_partial_rows(m, n);
  const size_t sums_at = c.take(dbias && sum_rows > 1 ? static_cast<size_t>(sum_rows) * n * 4 : 0);
  Input xi(a.x, m, k, a.ldx, dw, c), wi(a.w, n, k, a.ldw, dx, c);
  const float scale = drop.scale / dz_factor(a.act, dtype == OZ2_F16);  // 1 where dz is dy itself
  const Epilogue ep_dx = plain_epilogue(dx, a.lddx, m, k, scale, dtype), ep_dw = plain_epilogue(dw, a.lddw, n, k, scale, dtype);
  // the two products run side by side where they are small; else one after the other, and share the room for partial sums
  LinearPlan plan_dx, plan_dw;
  FewPlan pair{};
  if (dx) plan_dx = LinearPlan(Operand{nullptr, ld, false}, n, ep_dx, res.num_sms);
  if (dw) plan_dw = LinearPlan(Operand{nullptr, ld, true}, m, ep_dw, res.num_sms);
  if (dx && dw) pair = plan_few_pair(m, n, k, res.num_sms);
  const bool together = pair.ranks > 0 && pair.us < plan_dx.us + plan_dw.us;
  const size_t partial_at = c.take(together ? 0 : std::max(plan_dx.partial_bytes, plan_dw.partial_bytes));
  e = acquire_resources(st, c.used, &res);
  if (e != OZ2_OK) return e;
  if (make_dz || dbias) {
    DzArgs d{};
    d.m = m;
    d.n = n;
    d.dy = a.dy;
    d.lddy = a.lddy;
    d.preact = a.act == OZ2_ACT_NONE ? nullptr : a.preact;
    d.ldz = a.ldz;
    d.dz = make_dz ? res.workspace + dz_at : nullptr;
    d.lddz = ld;
    d.dbias = dbias;
    d.partial = sum_rows > 1 ? reinterpret_cast<float*>(res.workspace + sums_at) : nullptr;
    d.act = a.act;
    d.scale = scale;
    d.drop = drop;
    OZ2_TRY(launch_dz(d, dtype, st));
  }
  const void* dz = make_dz ? res.workspace + dz_at : a.dy;
  float* partial = reinterpret_cast<float*>(res.workspace + partial_at);
  const PackJob x_job = xi.place(res.workspace, a.ldx), w_job = wi.place(res.workspace, a.ldw);
  OZ2_TRY(launch_pack(x_job, w_job, st));
  if (together) {
    OZ2_TRY(launch_few_pair(pair, Operand{dz, ld, false}, Operand{wi.p, wi.ld, true}, Operand{xi.p, xi.ld, true}, ep_dx, ep_dw, dtype,
                            res, st));
    return OZ2_OK;
  }
  if (dx) OZ2_TRY(launch_linear(plan_dx, Operand{dz, ld, false}, Operand{wi.p, wi.ld, true}, n, ep_dx, dtype, res, partial, st));
  if (dw) OZ2_TRY(launch_linear(plan_dw, Operand{dz, ld, true}, Operand{xi.p, xi.ld, true}, m, ep_dw, dtype, res, partial, st));
  return OZ2_OK;
}

oz2_status dropout(const oz2_dropout_args& a, cudaStream_t st) {
  if (a.rows == 0 || a.cols == 0) return OZ2_OK;
  DeviceResources res;
  const oz2_status e = acquire_resources(st, 0, &res);
  if (e != OZ2_OK) return e;
  OZ2_TRY(launch_dropout(a.rows, a.cols, a.x, a.ldx, a.residual, a.ldr, a.y, a.ldy, static_cast<oz2_dtype>(a.dtype),
                         make_dropout(a.dropout, a.seed, a.offset), st));
  return OZ2_OK;
}

oz2_status qk(const oz2_qk_args& a, cudaStream_t st) {
  if (a.tokens == 0 || a.q.heads + a.k.heads == 0) return OZ2_OK;
  DeviceResources res;
  const oz2_status e = acquire_resources(st, 0, &res);
  if (e != OZ2_OK) return e;
  OZ2_TRY(launch_qk(a, res, st));
  return OZ2_OK;
}

oz2_status qk_backward(const oz2_qk_args& a, cudaStream_t st) {
  DeviceResources res;
  oz2_status e = acquire_resources(st, 0, &res);
  if (e != OZ2_OK) return e;
  if (a.tokens == 0 || a.q.heads + a.k.heads == 0) {  // sums over nothing
    const size_t bytes = a.dim * dtype_bytes(static_cast<oz2_dtype>(a.dtype));
    if (a.dq_weight) OZ2_TRY(cudaMemsetAsync(a.dq_weight, 0, bytes, st));
    if (a.dk_weight) OZ2_TRY(cudaMemsetAsync(a.dk_weight, 0, bytes, st));
    return OZ2_OK;
  }
  float* partial = nullptr;
  if (a.dq_weight || a.dk_weight) {
    e = acquire_resources(st, static_cast<size_t>(qk_partial_rows(a, res.num_sms)) * a.dim * 4, &res);
    if (e != OZ2_OK) return e;
    partial = reinterpret_cast<float*>(res.workspace);
  }
  OZ2_TRY(launch_qk_backward(a, res, partial, st));
  return OZ2_OK;
}

bool act_ok(int t) { return t >= OZ2_ACT_NONE && t <= OZ2_ACT_GELU_TANH; }

bool side_ok(const oz2_heads& h, int64_t tokens, int64_t heads) {
  return h.heads == heads && heads >= 0 && heads <= (1 << 20) && h.token_stride >= 0 && h.head_stride >= 0 &&
         (h.data != nullptr || heads == 0 || tokens == 0);
}

bool qk_ok(const oz2_qk_args& a) {
  return size_ok(a.tokens) && a.dim >= 1 && a.dim <= OZ2_HEAD_DIM_MAX && a.rot >= 0 && a.rot <= a.dim && a.rot % 2 == 0 &&
         dtype_ok(a.dtype) && side_ok(a.q, a.tokens, a.q.heads) && side_ok(a.k, a.tokens, a.k.heads) &&
         side_ok(a.q_out, a.tokens, a.q.heads) && side_ok(a.k_out, a.tokens, a.k.heads) &&
         (a.q_weight || a.q.heads == 0) && (a.k_weight || a.k.heads == 0) && a.eps >= 0.0 && a.table_rows >= 0 &&
         (a.rot == 0 || a.tokens == 0 || (a.positions && (a.table_rows == 0 || (a.cos && a.sin))));
}

}  // namespace
}  // namespace oz2

using namespace oz2;

extern "C" {

oz2_status ozaki2_linear(const oz2_linear_args* args, void* stream) {
  if (!args) return OZ2_ERR_INVALID_ARG;
  const oz2_linear_args& a = *args;
  if (!size_ok(a.m) || !size_ok(a.k) || !size_ok(a.n) || !is_16bit(a.dtype) || !act_ok(a.act) || !dropout_ok(a.dropout) ||
      !matrix_ok(a.x, a.m, a.k, a.ldx) || !matrix_ok(a.w, a.n, a.k, a.ldw) || !matrix_ok(a.y, a.m, a.n, a.ldy) ||
      (a.residual && a.ldr < a.n) || (a.preact && a.ldz < a.n))
    return OZ2_ERR_INVALID_ARG;
  return guarded([&] { return linear(a, static_cast<cudaStream_t>(stream)); });
}

oz2_status ozaki2_linear_backward(const oz2_linear_backward_args* args, void* stream) {
  if (!args) return OZ2_ERR_INVALID_ARG;
  const oz2_linear_backward_args& a = *args;
  if (!size_ok(a.m) || !size_ok(a.k) || !size_ok(a.n) || !is_16bit(a.dtype) || !act_ok(a.act) || !dropout_ok(a.dropout) ||
      !matrix_ok(a.dy, a.m, a.n, a.lddy) || (a.dw && !matrix_ok(a.x, a.m, a.k, a.ldx)) ||
      (a.dx && !matrix_ok(a.w, a.n, a.k, a.ldw)) || (a.act != OZ2_ACT_NONE && !matrix_ok(a.preact, a.m, a.n, a.ldz)) ||
      (a.dx && a.lddx < a.k) || (a.dw && a.lddw < a.k))
    return OZ2_ERR_INVALID_ARG;
  return guarded([&] { return linear_backward(a, static_cast<cudaStream_t>(stream)); });
}

oz2_status ozaki2_dropout(const oz2_dropout_args* args, void* stream) {
  if (!args) return OZ2_ERR_INVALID_ARG;
  const oz2_dropout_args& a = *args;
  if (!size_ok(a.rows) || !size_ok(a.cols) || !dtype_ok(a.dtype) || a.reserved != 0 || !dropout_ok(a.dropout) ||
      !matrix_ok(a.x, a.rows, a.cols, a.ldx) || !matrix_ok(a.y, a.rows, a.cols, a.ldy) || (a.residual && a.ldr < a.cols))
    return OZ2_ERR_INVALID_ARG;
  return guarded([&] { return dropout(a, static_cast<cudaStream_t>(stream)); });
}

oz2_status ozaki2_qk_norm_rope(const oz2_qk_args* args, void* stream) {
  if (!args || !qk_ok(*args)) return OZ2_ERR_INVALID_ARG;
  return guarded([&] { return qk(*args, static_cast<cudaStream_t>(stream)); });
}

oz2_status ozaki2_qk_norm_rope_backward(const oz2_qk_args* args, void* stream) {
  if (!args || !qk_ok(*args) || !side_ok(args->dq_out, args->tokens, args->q.heads) ||
      !side_ok(args->dk_out, args->tokens, args->k.heads))
    return OZ2_ERR_INVALID_ARG;
  return guarded([&] { return qk_backward(*args, static_cast<cudaStream_t>(stream)); });
}

}  // extern "C"
