// C ABI of the layer operators: argument checks, workspace and the choice of
// kernels.
#include <algorithm>
#include <cmath>
#include <new>

#include "oz2_layers.cuh"

namespace oz2 {
namespace {

#define OZ2_TRY(call)                                 \
  do {                                                \
    if ((call) != cudaSuccess) return OZ2_ERR_CUDA;   \
  } while (0)

bool is_16bit(int t) { return t == OZ2_BF16 || t == OZ2_F16; }
bool size_ok(int64_t n) { return n >= 0 && n <= OZ2_LAYER_DIM_MAX; }
// a matrix that a call reads or writes: present unless empty, rows that do not overlap
bool matrix_ok(const void* p, int64_t rows, int64_t cols, int64_t ld) {
  return ld >= cols && (p != nullptr || rows == 0 || cols == 0);
}
bool dropout_ok(double p) { return p >= 0.0 && p <= 1.0; }  // false for NaN

Dropout make_dropout(double p, uint64_t seed, uint64_t offset) {
  Dropout d;
  d.threshold = static_cast<uint32_t>(std::lround(65536.0 * p));
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
    copy = used && rows > 0 && cols > 0 && !aligned16(p, ld, OZ2_BF16);
    if (copy) {
      ld = ceil_div(cols, 8) * 8;
      at = c.take(static_cast<size_t>(rows) * ld * 2);
    }
  }
  // `from`'s leading dimension before the copy
  cudaError_t place(uint8_t* base, int64_t from_ld, cudaStream_t st) {
    if (!copy) return cudaSuccess;
    const void* from = p;
    p = base + at;
    return launch_pack(rows, cols, from, from_ld, base + at, ld, st);
  }
};

oz2_status linear(int64_t m, int64_t k, int64_t n, const void* x, int64_t ldx, const void* w, int64_t ldw, const void* bias,
                  const void* residual, int64_t ldr, void* y, int64_t ldy, void* preact, int64_t ldz, oz2_dtype dtype,
                  oz2_act act, double dropout, uint64_t seed, uint64_t offset, cudaStream_t st) {
  if (m == 0 || n == 0) return OZ2_OK;
  DeviceResources res;
  oz2_status e = acquire_resources(st, 0, &res);
  if (e != OZ2_OK) return e;
  Epilogue ep{};
  ep.bias = bias;
  ep.residual = residual;
  ep.y = y;
  ep.z = preact;
  ep.ldr = ldr;
  ep.ldy = ldy;
  ep.ldz = ldz;
  ep.rows = m;
  ep.cols = n;
  ep.act = act;
  ep.drop = make_dropout(dropout, seed, offset);
  ep.vec = aligned16(y, ldy, dtype) && (!bias || aligned16(bias, 0, dtype)) &&
           (!residual || aligned16(residual, ldr, dtype)) && (!preact || aligned16(preact, ldz, dtype));
  Carver c;
  Input xi(x, m, k, ldx, true, c), wi(w, n, k, ldw, true, c);
  const size_t partial = c.take(linear_workspace(k, ep, res.num_sms));
  e = acquire_resources(st, c.used, &res);
  if (e != OZ2_OK) return e;
  OZ2_TRY(xi.place(res.workspace, ldx, st));
  OZ2_TRY(wi.place(res.workspace, ldw, st));
  OZ2_TRY(launch_linear(Operand{xi.p, xi.ld, false}, Operand{wi.p, wi.ld, false}, k, ep, dtype, res,
                        reinterpret_cast<float*>(res.workspace + partial), st));
  return OZ2_OK;
}

// A plain product into out (no bias, activation, dropout or residual).
Epilogue plain_epilogue(void* out, int64_t ld, int64_t rows, int64_t cols, oz2_dtype dtype) {
  Epilogue ep{};
  ep.y = out;
  ep.ldy = ld;
  ep.rows = rows;
  ep.cols = cols;
  ep.vec = aligned16(out, ld, dtype);
  return ep;
}

oz2_status linear_backward(int64_t m, int64_t k, int64_t n, const void* dy, int64_t lddy, const void* x, int64_t ldx,
                           const void* w, int64_t ldw, const void* preact, int64_t ldz, void* dx, int64_t lddx, void* dw,
                           int64_t lddw, void* dbias, oz2_dtype dtype, oz2_act act, double dropout, uint64_t seed,
                           uint64_t offset, cudaStream_t st) {
  const Dropout drop = make_dropout(dropout, seed, offset);
  DeviceResources res;
  oz2_status e = acquire_resources(st, 0, &res);
  if (e != OZ2_OK) return e;
  // sums over nothing
  if (m == 0 || n == 0) {
    if (dx && m > 0 && k > 0) OZ2_TRY(cudaMemset2DAsync(dx, lddx * 2, 0, k * 2, m, st));
    if (dw && n > 0 && k > 0) OZ2_TRY(cudaMemset2DAsync(dw, lddw * 2, 0, k * 2, n, st));
    if (dbias && n > 0) OZ2_TRY(cudaMemsetAsync(dbias, 0, n * 2, st));
    return OZ2_OK;
  }
  if (k == 0) dx = dw = nullptr;
  // dz is dy itself where nothing follows the product and its rows are aligned
  const bool products = dx || dw;
  const bool make_dz = products && (act != OZ2_ACT_NONE || drop.threshold != 0 || !aligned16(dy, lddy, dtype));
  const int64_t ld = make_dz ? ceil_div(n, 8) * 8 : lddy;
  Carver c;
  const size_t dz_at = c.take(make_dz ? static_cast<size_t>(m) * ld * 2 : 0);
  const size_t sums_at = c.take(dbias ? static_cast<size_t>(dz_partial_rows(m, n)) * n * 4 : 0);
  Input xi(x, m, k, ldx, dw, c), wi(w, n, k, ldw, dx, c);
  const Epilogue ep_dx = plain_epilogue(dx, lddx, m, k, dtype), ep_dw = plain_epilogue(dw, lddw, n, k, dtype);
  // the two products run one after the other and share the room for partial sums
  const size_t partial_at = c.take(std::max(dx ? linear_workspace(n, ep_dx, res.num_sms) : 0,
                                            dw ? linear_workspace(m, ep_dw, res.num_sms) : 0));
  e = acquire_resources(st, c.used, &res);
  if (e != OZ2_OK) return e;
  if (make_dz || dbias) {
    DzArgs a{};
    a.m = m;
    a.n = n;
    a.dy = dy;
    a.lddy = lddy;
    a.preact = preact;
    a.ldz = ldz;
    a.dz = make_dz ? res.workspace + dz_at : nullptr;
    a.lddz = ld;
    a.dbias = dbias;
    a.partial = reinterpret_cast<float*>(res.workspace + sums_at);
    a.act = act;
    a.drop = drop;
    OZ2_TRY(launch_dz(a, dtype, st));
  }
  const void* dz = make_dz ? res.workspace + dz_at : dy;
  float* partial = reinterpret_cast<float*>(res.workspace + partial_at);
  OZ2_TRY(xi.place(res.workspace, ldx, st));
  OZ2_TRY(wi.place(res.workspace, ldw, st));
  if (dx) OZ2_TRY(launch_linear(Operand{dz, ld, false}, Operand{wi.p, wi.ld, true}, n, ep_dx, dtype, res, partial, st));
  if (dw) OZ2_TRY(launch_linear(Operand{dz, ld, true}, Operand{xi.p, xi.ld, true}, m, ep_dw, dtype, res, partial, st));
  return OZ2_OK;
}

bool side_ok(const oz2_heads& h, int64_t tokens, int64_t heads) {
  return h.heads == heads && heads >= 0 && heads <= (1 << 20) && h.token_stride >= 0 && h.head_stride >= 0 &&
         (h.data != nullptr || heads == 0 || tokens == 0);
}

bool qk_ok(const QkArgs& a, double eps, int dtype) {
  return size_ok(a.tokens) && a.dim >= 1 && a.dim <= OZ2_HEAD_DIM_MAX && a.rot >= 0 && a.rot <= a.dim && a.rot % 2 == 0 &&
         dtype >= OZ2_BF16 && dtype <= OZ2_F32 && side_ok(a.q, a.tokens, a.q.heads) && side_ok(a.k, a.tokens, a.k.heads) &&
         side_ok(a.q_out, a.tokens, a.q.heads) && side_ok(a.k_out, a.tokens, a.k.heads) &&
         (a.q_weight || a.q.heads == 0) && (a.k_weight || a.k.heads == 0) && eps >= 0.0 && a.table_rows >= 0 &&
         (a.rot == 0 || a.tokens == 0 || (a.cos && a.sin && a.positions));
}

// No exception leaves a C entry point; what can be thrown is the host's own lack of memory.
template <typename F>
oz2_status guarded(F&& f) {
  try {
    std::lock_guard<std::mutex> lk(library_mutex());
    return f();
  } catch (const std::bad_alloc&) {
    return OZ2_ERR_NO_MEMORY;
  } catch (...) {
    return OZ2_ERR_CUDA;
  }
}

}  // namespace
}  // namespace oz2

using namespace oz2;

extern "C" {

oz2_status ozaki2_linear(int64_t m, int64_t k, int64_t n, const void* x, int64_t ldx, const void* w, int64_t ldw,
                         const void* bias, const void* residual, int64_t ldr, void* y, int64_t ldy, void* preact,
                         int64_t ldz, oz2_dtype dtype, oz2_act act, double dropout, uint64_t seed, uint64_t offset,
                         void* stream) {
  if (!size_ok(m) || !size_ok(k) || !size_ok(n) || !is_16bit(dtype) || act < OZ2_ACT_NONE || act > OZ2_ACT_GELU_TANH ||
      !dropout_ok(dropout) || !matrix_ok(x, m, k, ldx) || !matrix_ok(w, n, k, ldw) || !matrix_ok(y, m, n, ldy) ||
      (residual && ldr < n) || (preact && ldz < n))
    return OZ2_ERR_INVALID_ARG;
  return guarded([&] {
    return linear(m, k, n, x, ldx, w, ldw, bias, residual, ldr, y, ldy, preact, ldz, dtype, act, dropout, seed, offset,
                  static_cast<cudaStream_t>(stream));
  });
}

oz2_status ozaki2_linear_backward(int64_t m, int64_t k, int64_t n, const void* dy, int64_t lddy, const void* x,
                                  int64_t ldx, const void* w, int64_t ldw, const void* preact, int64_t ldz, void* dx,
                                  int64_t lddx, void* dw, int64_t lddw, void* dbias, oz2_dtype dtype, oz2_act act,
                                  double dropout, uint64_t seed, uint64_t offset, void* stream) {
  if (!size_ok(m) || !size_ok(k) || !size_ok(n) || !is_16bit(dtype) || act < OZ2_ACT_NONE || act > OZ2_ACT_GELU_TANH ||
      !dropout_ok(dropout) || !matrix_ok(dy, m, n, lddy) || (dw && !matrix_ok(x, m, k, ldx)) ||
      (dx && !matrix_ok(w, n, k, ldw)) || (act != OZ2_ACT_NONE && !matrix_ok(preact, m, n, ldz)) || (dx && lddx < k) ||
      (dw && lddw < k))
    return OZ2_ERR_INVALID_ARG;
  return guarded([&] {
    return linear_backward(m, k, n, dy, lddy, x, ldx, w, ldw, act == OZ2_ACT_NONE ? nullptr : preact, ldz, dx, lddx, dw,
                           lddw, dbias, dtype, act, dropout, seed, offset, static_cast<cudaStream_t>(stream));
  });
}

oz2_status ozaki2_dropout(int64_t rows, int64_t cols, const void* x, int64_t ldx, const void* residual, int64_t ldr,
                          void* y, int64_t ldy, oz2_dtype dtype, double dropout, uint64_t seed, uint64_t offset,
                          void* stream) {
  if (!size_ok(rows) || !size_ok(cols) || dtype < OZ2_BF16 || dtype > OZ2_F32 || !dropout_ok(dropout) ||
      !matrix_ok(x, rows, cols, ldx) || !matrix_ok(y, rows, cols, ldy) || (residual && ldr < cols))
    return OZ2_ERR_INVALID_ARG;
  return guarded([&] {
    if (rows == 0 || cols == 0) return OZ2_OK;
    DeviceResources res;
    const oz2_status e = acquire_resources(static_cast<cudaStream_t>(stream), 0, &res);
    if (e != OZ2_OK) return e;
    OZ2_TRY(launch_dropout(rows, cols, x, ldx, residual, ldr, y, ldy, dtype, make_dropout(dropout, seed, offset),
                           static_cast<cudaStream_t>(stream)));
    return OZ2_OK;
  });
}

oz2_status ozaki2_qk_norm_rope(int64_t tokens, int64_t dim, int64_t rot, oz2_heads q, oz2_heads k, const void* q_weight,
                               const void* k_weight, const float* cos, const float* sin, int64_t table_rows,
                               const int64_t* positions, double eps, int interleaved, oz2_dtype dtype, oz2_heads q_out,
                               oz2_heads k_out, void* stream) {
  if (dim < 0 || dim > OZ2_HEAD_DIM_MAX || rot < 0 || rot > dim) return OZ2_ERR_INVALID_ARG;
  QkArgs a{};
  a.tokens = tokens;
  a.dim = static_cast<int>(dim);
  a.rot = static_cast<int>(rot);
  a.q = q;
  a.k = k;
  a.q_out = q_out;
  a.k_out = k_out;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.cos = cos;
  a.sin = sin;
  a.table_rows = table_rows;
  a.positions = positions;
  a.eps = static_cast<float>(eps);
  a.interleaved = interleaved != 0;
  if (!qk_ok(a, eps, dtype)) return OZ2_ERR_INVALID_ARG;
  return guarded([&] {
    if (tokens == 0 || q.heads + k.heads == 0) return OZ2_OK;
    DeviceResources res;
    const oz2_status e = acquire_resources(static_cast<cudaStream_t>(stream), 0, &res);
    if (e != OZ2_OK) return e;
    OZ2_TRY(launch_qk(a, dtype, static_cast<cudaStream_t>(stream)));
    return OZ2_OK;
  });
}

oz2_status ozaki2_qk_norm_rope_backward(int64_t tokens, int64_t dim, int64_t rot, oz2_heads dq_out, oz2_heads dk_out,
                                        oz2_heads q, oz2_heads k, const void* q_weight, const void* k_weight,
                                        const float* cos, const float* sin, int64_t table_rows,
                                        const int64_t* positions, double eps, int interleaved, oz2_dtype dtype,
                                        oz2_heads dq, oz2_heads dk, void* dq_weight, void* dk_weight, void* stream) {
  if (dim < 0 || dim > OZ2_HEAD_DIM_MAX || rot < 0 || rot > dim) return OZ2_ERR_INVALID_ARG;
  QkArgs a{};
  a.tokens = tokens;
  a.dim = static_cast<int>(dim);
  a.rot = static_cast<int>(rot);
  a.q = q;
  a.k = k;
  a.q_out = dq;
  a.k_out = dk;
  a.dq_out = dq_out;
  a.dk_out = dk_out;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.cos = cos;
  a.sin = sin;
  a.table_rows = table_rows;
  a.positions = positions;
  a.eps = static_cast<float>(eps);
  a.interleaved = interleaved != 0;
  a.dq_weight = dq_weight;
  a.dk_weight = dk_weight;
  if (!qk_ok(a, eps, dtype) || !side_ok(dq_out, tokens, q.heads) || !side_ok(dk_out, tokens, k.heads))
    return OZ2_ERR_INVALID_ARG;
  return guarded([&] {
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool none = tokens == 0 || q.heads + k.heads == 0, weights = dq_weight || dk_weight;
    DeviceResources res;
    oz2_status e = acquire_resources(st, 0, &res);
    if (e != OZ2_OK) return e;
    if (none) {
      if (dq_weight) OZ2_TRY(cudaMemsetAsync(dq_weight, 0, dim * dtype_bytes(dtype), st));
      if (dk_weight) OZ2_TRY(cudaMemsetAsync(dk_weight, 0, dim * dtype_bytes(dtype), st));
      return OZ2_OK;
    }
    const int64_t rows = qk_partial_rows(tokens, q.heads + k.heads, res.num_sms);
    if (weights) {
      e = acquire_resources(st, static_cast<size_t>(rows) * 2 * dim * 4, &res);
      if (e != OZ2_OK) return e;
      a.partial = reinterpret_cast<float*>(res.workspace);
    }
    OZ2_TRY(launch_qk_backward(a, dtype, rows, st));
    return OZ2_OK;
  });
}

}  // extern "C"
