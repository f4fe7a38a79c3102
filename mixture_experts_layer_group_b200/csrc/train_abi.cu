// C ABI of the layer's backward steps (declared in include/moe_b200.h):
// argument checks, workspace carving and launch sequences, all on the
// caller's stream. The training forward lives with the forward (moe_abi.cu),
// the gradient norm and clipping in grad_clip.cu.
#include "internal.h"

namespace moe {
namespace {

struct BwdLayout {
  size_t status, sched, grp_row0, grp_rows, unit_base1, unit_base2;
  size_t dg, du, gh, part;
  size_t total;
};

BwdLayout make_bwd_layout(const Problem& p) {
  BwdLayout L{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    size_t at = off;
    off = align256(off + bytes);
    return at;
  };
  const size_t N = (size_t)p.N, rf = (size_t)p.R * p.F * p.elem;
  L.status = take(256);  // first, as in every workspace of the library
  L.sched = take(256);
  L.grp_row0 = take((N + 1) * 4);
  L.grp_rows = take((N + 1) * 4);
  L.unit_base1 = take((N + 2) * 4);
  L.unit_base2 = take((N + 2) * 4);
  L.dg = take(rf);
  L.du = take(rf);
  L.gh = take(rf);
  // (narrowest tiles: a workspace for R rows also holds a call of fewer)
  L.part = take((size_t)((p.F + 31) / 32) * p.R * 4);
  L.total = off;
  return L;
}

// The router's products: row tables, the logits' gradient (fp32, or bf16 by
// token and by expert) and the planes of a split weight gradient.
struct RouteLayout {
  size_t status, tables, dz, dz_t, planes;
  size_t total;
  int splits;
  int64_t ld, ld_t;
};

RouteLayout make_route_layout(const Problem& p) {
  RouteLayout L{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    size_t at = off;
    off = align256(off + bytes);
    return at;
  };
  const bool tc = p.dtype == MOE_BF16;
  L.ld = (p.N + 7) / 8 * 8;
  L.ld_t = (p.T + 7) / 8 * 8;
  L.splits = 1;
  int64_t planes = 1;
  if (tc) {
    const RoutePlan plan = plan_route_products(p);
    L.splits = plan.splits;
    planes = plan.most_splits;  // (a workspace for T tokens also holds a call of fewer)
  } else {
    // dW_r is N x d summed over all tokens, few tiles with a long sum: the tokens
    // are split so that there are about four tiles of 64 x 64 per SM
    const int64_t tiles = (int64_t)((p.N + 63) / 64) * ((p.d + 63) / 64);
    planes = 4 * kRouterTargetSms / tiles;
    if (planes > p.T / 64) planes = p.T / 64;
    if (planes > kMaxRouteSplits) planes = kMaxRouteSplits;
    if (planes > 1) L.splits = (int)planes;
  }
  L.status = take(256);
  L.tables = take(kRouteTables * 4);
  L.dz = take((size_t)p.T * L.ld * p.elem);
  L.dz_t = take(tc ? (size_t)p.N * L.ld_t * 2 : 0);
  L.planes = take(planes > 1 ? (size_t)planes * p.N * p.d * 4 : 0);
  L.total = off;
  return L;
}

// The weight gradients' type and whether they are added to.
moe_status check_grad(const Problem& p, int32_t grad_dtype, int32_t accumulate) {
  if (grad_dtype != MOE_F32 && grad_dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (grad_dtype == MOE_BF16 && p.dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  // a bf16 sum over steps loses what each step adds: fp32 only
  if (accumulate && grad_dtype != MOE_F32) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

bool bad4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

moe_status check_workspace(const void* ws, size_t have, size_t need) {
  return !ws || have < need || (reinterpret_cast<uintptr_t>(ws) & 255u) ? MOE_ERR_WORKSPACE : MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_experts_backward_workspace_size(const moe_cfg* cfg, int64_t rows, size_t* bytes) {
  Problem p;
  moe_status st = make_group_problem(cfg, rows, &p);
  if (st != MOE_OK) return st;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = make_bwd_layout(p).total;
  return MOE_OK;
}

moe_status moe_experts_backward(const moe_cfg* cfg, int64_t rows, const int32_t* counts, const void* x_rows,
                                const float* gate_rows, const void* W1, const void* W3, const void* W2,
                                const void* gu, const void* dy_rows, void* dx_rows, float* dgate_rows, void* dW1,
                                void* dW3, void* dW2, int32_t grad_dtype, int32_t accumulate, void* ws,
                                size_t ws_bytes, void* stream) {
  Problem p;
  moe_status st = make_group_problem(cfg, rows, &p);
  if (st != MOE_OK) return st;
  if ((st = check_grad(p, grad_dtype, accumulate)) != MOE_OK) return st;
  const bool any_dw = dW1 || dW3 || dW2;
  if (any_dw && (!dW1 || !dW3 || !dW2 || !aligned16(dW1) || !aligned16(dW3) || !aligned16(dW2)))
    return MOE_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  if (rows == 0) {
    // no rows: the weight gradients are zero (or unchanged)
    if (!any_dw || accumulate) return MOE_OK;
    const size_t n = (size_t)p.N * p.F * p.d * (grad_dtype == MOE_F32 ? 4 : 2);
    cudaError_t e = cudaMemsetAsync(dW1, 0, n, s);
    if (e == cudaSuccess) e = cudaMemsetAsync(dW3, 0, n, s);
    if (e == cudaSuccess) e = cudaMemsetAsync(dW2, 0, n, s);
    return e == cudaSuccess ? MOE_OK : cuda_fail(e);
  }
  if (!counts || !x_rows || !W1 || !W3 || !W2 || !gu || !dy_rows) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x_rows) || !aligned16(W1) || !aligned16(W3) || !aligned16(W2) || !aligned16(gu) ||
      !aligned16(dy_rows) || !aligned16(dx_rows) || bad4(counts) || bad4(gate_rows) || bad4(dgate_rows))
    return MOE_ERR_INVALID_ARG;
  const BwdLayout L = make_bwd_layout(p);
  if ((st = check_workspace(ws, ws_bytes, L.total)) != MOE_OK) return st;
  unsigned* status = at<unsigned>(ws, L.status);
  cudaError_t e = wait_host_outputs(ws, s);
  if (e != cudaSuccess) return cuda_fail(e);
  DispatchBuffers db{};
  db.status = status;
  db.grp_row0 = at<int32_t>(ws, L.grp_row0);
  db.grp_rows = at<int32_t>(ws, L.grp_rows);
  db.unit_base1 = at<int32_t>(ws, L.unit_base1);
  db.unit_base2 = at<int32_t>(ws, L.unit_base2);
  const bool tc = p.dtype == MOE_BF16;
  const int bs = tc ? 0 : simt_bwd_tile(p), bc = simt_cols(bs);
  e = launch_group_tables(p, counts, db, tc ? kTcBM : bs, tc ? dh_tile(p) : bc, tc ? kTcBN2 : bc,
                          at<int>(ws, L.sched), s);
  if (e != cudaSuccess) return cuda_fail(e);
  ExpertsBwdArgs a{};
  a.x_rows = x_rows;
  a.gate_rows = gate_rows;
  a.W1 = W1;
  a.W3 = W3;
  a.W2 = W2;
  a.gu = gu;
  a.dy_rows = dy_rows;
  a.dx_rows = dx_rows;
  a.dgate_rows = dgate_rows;
  a.dW1 = dW1;
  a.dW3 = dW3;
  a.dW2 = dW2;
  a.grad_dtype = grad_dtype;
  a.accumulate = accumulate != 0;
  a.dg = at<void>(ws, L.dg);
  a.du = at<void>(ws, L.du);
  a.gh = at<void>(ws, L.gh);
  a.dgate_part = at<float>(ws, L.part);
  a.grp_row0 = db.grp_row0;
  a.grp_rows = db.grp_rows;
  a.unit_base1 = db.unit_base1;
  a.unit_base2 = db.unit_base2;
  a.status = status;
  a.sched = at<int>(ws, L.sched);
  e = tc ? launch_experts_backward_tc(p, a, s) : launch_experts_backward_simt(p, a, s);
  if (e == cudaSuccess) e = note_device_use(ws, s);
  return e == cudaSuccess ? MOE_OK : cuda_fail(e);
}

moe_status moe_combine_backward(const moe_cfg* cfg, int64_t T, const void* dy, const int32_t* slot_pos,
                                void* dy_rows, void* stream) {
  Problem p;
  moe_status st = make_problem(cfg, T, &p);
  if (st != MOE_OK) return st;
  if (T == 0) return MOE_OK;
  if (!dy || !slot_pos || !dy_rows || !aligned16(dy) || !aligned16(dy_rows) || bad4(slot_pos))
    return MOE_ERR_INVALID_ARG;
  const cudaError_t e = launch_gather(p, dy, slot_pos, dy_rows, nullptr, (cudaStream_t)stream);
  return e == cudaSuccess ? MOE_OK : cuda_fail(e);
}

moe_status moe_dispatch_backward(const moe_cfg* cfg, int64_t T, const void* dx_rows, const int32_t* slot_pos,
                                 const void* dx_shared, const void* dx_router, void* dx, void* stream) {
  Problem p;
  moe_status st = make_problem(cfg, T, &p);
  if (st != MOE_OK) return st;
  if (T == 0) return MOE_OK;
  if (!dx_rows || !slot_pos || !dx || !aligned16(dx_rows) || !aligned16(dx) || !aligned16(dx_shared) ||
      !aligned16(dx_router) || bad4(slot_pos))
    return MOE_ERR_INVALID_ARG;
  const cudaError_t e = launch_combine_rows(p, dx_rows, dx_shared, slot_pos, dx, (cudaStream_t)stream, dx_router);
  return e == cudaSuccess ? MOE_OK : cuda_fail(e);
}

moe_status moe_route_backward_workspace_size(const moe_cfg* cfg, int64_t T, size_t* bytes) {
  Problem p;
  moe_status st = make_problem(cfg, T, &p);
  if (st != MOE_OK) return st;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = make_route_layout(p).total;
  return MOE_OK;
}

moe_status moe_route_backward(const moe_cfg* cfg, int64_t T, const void* x, const void* W_r, const float* logits,
                              const int32_t* topk_idx, const float* dgates, const int32_t* slot_pos, void* dx,
                              void* dW_r, int32_t grad_dtype, int32_t accumulate, void* ws, size_t ws_bytes,
                              void* stream) {
  Problem p;
  moe_status st = make_problem(cfg, T, &p);
  if (st != MOE_OK) return st;
  if ((st = check_grad(p, grad_dtype, accumulate)) != MOE_OK) return st;
  if (!aligned16(dW_r)) return MOE_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  if (T == 0) {
    if (!dW_r || accumulate) return MOE_OK;
    const cudaError_t e = cudaMemsetAsync(dW_r, 0, (size_t)p.N * p.d * (grad_dtype == MOE_F32 ? 4 : 2), s);
    return e == cudaSuccess ? MOE_OK : cuda_fail(e);
  }
  if (!x || !W_r || !logits || !topk_idx || !dgates || !aligned16(x) || !aligned16(W_r) || !aligned16(dx) ||
      bad4(logits) || bad4(topk_idx) || bad4(dgates) || bad4(slot_pos))
    return MOE_ERR_INVALID_ARG;
  const RouteLayout L = make_route_layout(p);
  if ((st = check_workspace(ws, ws_bytes, L.total)) != MOE_OK) return st;
  unsigned* status = at<unsigned>(ws, L.status);
  cudaError_t e = wait_host_outputs(ws, s);
  if (e == cudaSuccess) e = cudaMemsetAsync(status, 0, 4, s);
  if (e != cudaSuccess) return cuda_fail(e);
  const bool tc = p.dtype == MOE_BF16;
  Problem one = p;  // the products' one group of T rows
  one.F = p.d;
  one.N = 1;
  one.R = T;
  const int bs = simt_bwd_tile(one), bc = simt_cols(bs);
  const int64_t units = (T + bs - 1) / bs * ((p.d + bc - 1) / bc);  // fp32 row tiles
  if (units > (1ll << 31) - 1) return MOE_ERR_UNSUPPORTED;
  RouteDzArgs z{};
  z.logits = logits;
  z.idx = topk_idx;
  z.dgates = dgates;
  z.slot_pos = slot_pos;
  z.T = T;
  z.N = p.N;
  z.k = p.k;
  z.score_fn = p.score_fn;
  z.normalize = p.normalize;
  z.route_scale = p.route_scale;
  z.status = status;
  z.dz = tc ? nullptr : at<float>(ws, L.dz);
  z.dz16 = at<__nv_bfloat16>(ws, L.dz);
  z.dz16_t = tc && dx ? at<__nv_bfloat16>(ws, L.dz_t) : nullptr;
  z.ld = L.ld;
  z.ld_t = L.ld_t;
  z.tables = at<int32_t>(ws, L.tables);
  int32_t* v = z.table_values;
  v[kRtRows] = (int32_t)T;
  v[kRtUnits + 1] = v[kRtUnits + 2] = (int32_t)units;
  v[kRtExperts] = p.N;
  for (int i = 0; i < L.splits; ++i) {
    const int64_t lo = T * i / L.splits / 64 * 64, hi = i + 1 == L.splits ? T : T * (i + 1) / L.splits / 64 * 64;
    v[kRtSplit0 + i] = (int32_t)lo;
    v[kRtSplitRows + i] = (int32_t)(hi - lo);
  }
  if ((e = launch_route_dz(z, s)) != cudaSuccess) return cuda_fail(e);
  RouteBwdArgs a{};
  a.x = x;
  a.W_r = W_r;
  a.dx = dx;
  a.dW_r = dW_r;
  a.grad_dtype = grad_dtype;
  a.accumulate = accumulate != 0;
  a.status = status;
  a.dz = z.dz;
  a.dz16 = z.dz16;
  a.dz16_t = z.dz16_t;
  a.ld = L.ld;
  a.ld_t = L.ld_t;
  a.tables = z.tables;
  a.splits = L.splits;
  a.planes = at<float>(ws, L.planes);
  e = tc ? launch_route_products_tc(p, a, s) : launch_route_products_simt(p, a, s);
  if (e == cudaSuccess) e = note_device_use(ws, s);
  return e == cudaSuccess ? MOE_OK : cuda_fail(e);
}

}  // extern "C"
