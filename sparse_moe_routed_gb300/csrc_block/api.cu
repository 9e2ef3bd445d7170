// extern "C" boundary of libmoe_block: host-side admission of every argument,
// then the kernel launches on the caller's stream.  Nothing is enqueued and
// nothing is written unless every check passes (AFN-010 "One bank flip is
// enough: make the whole inference chunk transactional", section "The
// publication model"; AFN-001, section "Phase 3: reject before the GPU
// exists").  Declarations and argument contracts: include/moe_block.h.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "../csrc/common.cuh"
#include "launch.h"

namespace moe {
namespace blk {

int sm_count() {
  static std::atomic<int> cache[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
  int v = cache[dev].load(std::memory_order_relaxed);
  if (v > 0) return v;
  if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v < 1) return 1;
  cache[dev].store(v, std::memory_order_relaxed);
  return v;
}

}  // namespace blk
}  // namespace moe

namespace {

using moe::blk::Rows;

constexpr int kMaxH = 65536;      // the row movements
constexpr int kMaxNormH = 16384;  // the norms
constexpr int kMaxT = 1 << 30;    // tokens: launch sizes are computed in int

inline bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool a4(const void* p) { return aligned(p, 4); }
inline bool type_ok(int t) { return t == MOE_ROW_F32 || t == MOE_ROW_BF16; }
inline unsigned width(int t) { return t == MOE_ROW_F32 ? 4 : 2; }

inline Rows rows(const void* p, int64_t ld, int type) { return Rows{const_cast<void*>(p), ld, type}; }

// n rows of H elements.  Null rows pass here: a call says which it needs.
inline moe_status check_rows(const Rows& r, int64_t n, int H) {
  if (r.p == nullptr) return MOE_OK;
  if (!aligned(r.p, width(r.type))) return MOE_EINVAL;
  if (r.ld < H) return MOE_ESHAPE;
  if (n > 0 && r.ld > (INT64_MAX / 8) / n) return MOE_ENOTSUP;
  return MOE_OK;
}

inline moe_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ECUDA; }

#define MOE_TRY(expr)                 \
  do {                                \
    const moe_status s_ = (expr);     \
    if (s_ != MOE_OK) return s_;      \
  } while (0)

moe_status check_routes(int T, int k, int H, int R, const int32_t* slots, const float* w, const int32_t* status) {
  if (T < 0 || k <= 0 || H <= 0 || R < 0) return MOE_ESHAPE;
  if (k > moe::kMaxK || H > kMaxH || T > kMaxT || static_cast<long long>(T) * k >= (1LL << 31)) return MOE_ENOTSUP;
  if (T > 0 && !slots) return MOE_EINVAL;
  if (!a4(slots) || !a4(w) || !a4(status)) return MOE_EINVAL;
  return MOE_OK;
}

}  // namespace

extern "C" {

int moe_block_abi_version(void) { return 100; }

moe_status moe_dispatch(const void* x, int64_t ldx, int row_type, const int32_t* inv_perm, const float* w, int T,
                        int k, int H, int R, void* x_perm, int64_t ld_perm, int32_t* dev_status, void* stream) {
  if (!type_ok(row_type)) return MOE_EINVAL;
  MOE_TRY(check_routes(T, k, H, R, inv_perm, w, dev_status));
  const Rows rx = rows(x, ldx, row_type), rp = rows(x_perm, ld_perm, row_type);
  MOE_TRY(check_rows(rx, T, H));
  MOE_TRY(check_rows(rp, R, H));
  if (T == 0) return MOE_OK;
  if (!x || (R > 0 && !x_perm) || x == x_perm) return MOE_EINVAL;
  return cuda_status(moe::blk::launch_spread(rx, rows(nullptr, 0, row_type), inv_perm, w, T, k, H, R, rp, nullptr,
                                             dev_status, static_cast<cudaStream_t>(stream)));
}

moe_status moe_dispatch_backward(const void* dx_perm, int64_t ld_perm, int row_type, const int32_t* inv_perm,
                                 const float* w, const void* x, int64_t ldx, int T, int k, int H, int R, void* dx,
                                 int64_t ldx_grad, int dx_type, const void* add, int64_t ld_add, float* dw,
                                 int32_t* dev_status, void* stream) {
  if (!type_ok(row_type) || !type_ok(dx_type)) return MOE_EINVAL;
  MOE_TRY(check_routes(T, k, H, R, inv_perm, w, dev_status));
  const Rows rp = rows(dx_perm, ld_perm, row_type), rx = rows(dw ? x : nullptr, ldx, row_type),
             rd = rows(dx, ldx_grad, dx_type), ra = rows(add, ld_add, dx_type);
  MOE_TRY(check_rows(rp, R, H));
  MOE_TRY(check_rows(rx, T, H));
  MOE_TRY(check_rows(rd, T, H));
  MOE_TRY(check_rows(ra, T, H));
  if (T == 0) return MOE_OK;
  if ((R > 0 && !dx_perm) || !dx || (dw && !x) || !a4(dw)) return MOE_EINVAL;
  if (dx == dx_perm || (dw && dx == x) || (add == dx && ld_add != ldx_grad)) return MOE_EINVAL;
  return cuda_status(moe::blk::launch_join(rp, rx, inv_perm, w, T, k, H, R, rd, ra, dw, dev_status,
                                           static_cast<cudaStream_t>(stream)));
}

moe_status moe_collect(const void* y_perm, int64_t ld_perm, int row_type, const int32_t* inv_perm, const float* w,
                       int T, int k, int H, int R, void* out, int64_t ld_out, int out_type, const void* add,
                       int64_t ld_add, int32_t* dev_status, void* stream) {
  if (!type_ok(row_type) || !type_ok(out_type)) return MOE_EINVAL;
  MOE_TRY(check_routes(T, k, H, R, inv_perm, w, dev_status));
  const Rows rp = rows(y_perm, ld_perm, row_type), ro = rows(out, ld_out, out_type),
             ra = rows(add, ld_add, out_type);
  MOE_TRY(check_rows(rp, R, H));
  MOE_TRY(check_rows(ro, T, H));
  MOE_TRY(check_rows(ra, T, H));
  if (T == 0) return MOE_OK;
  if ((R > 0 && !y_perm) || !out || out == y_perm || (add == out && ld_add != ld_out)) return MOE_EINVAL;
  return cuda_status(moe::blk::launch_join(rp, rows(nullptr, 0, row_type), inv_perm, w, T, k, H, R, ro, ra, nullptr,
                                           dev_status, static_cast<cudaStream_t>(stream)));
}

moe_status moe_collect_backward(const void* dout, int64_t ld_dout, int out_type, const void* y_perm, int64_t ld_perm,
                                int row_type, const int32_t* inv_perm, const float* w, int T, int k, int H, int R,
                                void* dy_perm, int64_t ld_dperm, float* dw, int32_t* dev_status, void* stream) {
  if (!type_ok(row_type) || !type_ok(out_type)) return MOE_EINVAL;
  MOE_TRY(check_routes(T, k, H, R, inv_perm, w, dev_status));
  const Rows ro = rows(dout, ld_dout, out_type), ry = rows(dw ? y_perm : nullptr, ld_perm, row_type),
             rd = rows(dy_perm, ld_dperm, row_type);
  MOE_TRY(check_rows(ro, T, H));
  MOE_TRY(check_rows(ry, R, H));
  MOE_TRY(check_rows(rd, R, H));
  if (T == 0) return MOE_OK;
  if (!dout || (R > 0 && !dy_perm) || (dw && R > 0 && !y_perm) || !a4(dw)) return MOE_EINVAL;
  if (dy_perm == dout || (dw && R > 0 && dy_perm == y_perm)) return MOE_EINVAL;
  return cuda_status(moe::blk::launch_spread(ro, ry, inv_perm, w, T, k, H, R, rd, dw, dev_status,
                                             static_cast<cudaStream_t>(stream)));
}

// What both directions of the block norm have in common.
static moe_status check_norm(int x_type, const void* y, int y_type, const void* gate, int gate_kind, int64_t ld_gate,
                             const float* gamma_post, const float* gamma_pre, int post_norm, float scale, int T,
                             int H) {
  if (T < 0 || H <= 0) return MOE_ESHAPE;
  if (H > kMaxNormH || T > kMaxT) return MOE_ENOTSUP;
  if (!type_ok(x_type) || !type_ok(y_type)) return MOE_EINVAL;
  if (gate_kind < MOE_GATE_NONE || gate_kind > MOE_GATE_FULL) return MOE_EINVAL;
  if ((gate_kind == MOE_GATE_NONE) != (gate == nullptr) && !(T == 0 && gate_kind >= MOE_GATE_TOKEN))
    return MOE_EINVAL;
  if (gate_kind == MOE_GATE_FULL)
    MOE_TRY(check_rows(rows(gate, ld_gate, y_type), T, H));
  else if (!a4(gate))
    return MOE_EINVAL;
  if (!a4(gamma_post) || !a4(gamma_pre) || !std::isfinite(scale)) return MOE_EINVAL;
  if (gamma_post && !post_norm) return MOE_EINVAL;
  if (T > 0 && !y && (post_norm || gate_kind != MOE_GATE_NONE)) return MOE_EINVAL;
  return MOE_OK;
}

moe_status moe_block_norm(const void* x, int64_t ldx, int x_type, const void* y, int64_t ldy, int y_type,
                          const void* gate, int gate_kind, int64_t ld_gate, const float* gamma_post,
                          const float* gamma_pre, int post_norm, float scale, float eps, int T, int H, void* x_out,
                          int64_t ldx_out, void* n_out, int64_t ldn, float* rstd_post, float* rstd_pre,
                          void* stream) {
  MOE_TRY(check_norm(x_type, y, y_type, gate, gate_kind, ld_gate, gamma_post, gamma_pre, post_norm, scale, T, H));
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return MOE_EINVAL;
  moe::blk::NormArgs a{};
  a.x = rows(x, ldx, x_type);
  a.y = rows(y, ldy, y_type);
  a.gate = rows(gate, gate_kind == MOE_GATE_FULL ? ld_gate : 0, y_type);
  a.x_out = rows(x_out, ldx_out, x_type);
  a.n_out = rows(n_out, ldn, y_type);
  MOE_TRY(check_rows(a.x, T, H));
  MOE_TRY(check_rows(a.y, T, H));
  MOE_TRY(check_rows(a.x_out, T, H));
  MOE_TRY(check_rows(a.n_out, T, H));
  if (!a4(rstd_post) || !a4(rstd_pre)) return MOE_EINVAL;
  if (T == 0) return MOE_OK;
  if (!x || (!x_out && !n_out)) return MOE_EINVAL;
  if ((rstd_post && !post_norm) || (!n_out && (gamma_pre || rstd_pre))) return MOE_EINVAL;
  if ((x_out == x && ldx_out != ldx) || (x_out && (x_out == y || x_out == n_out)) ||
      (n_out && (n_out == x || n_out == y)))
    return MOE_EINVAL;
  a.gate_kind = gate_kind;
  a.post_norm = post_norm != 0;
  a.gamma_post = gamma_post;
  a.gamma_pre = gamma_pre;
  a.scale = scale;
  a.eps = eps;
  a.T = T;
  a.H = H;
  a.rstd_post = rstd_post;
  a.rstd_pre = rstd_pre;
  return cuda_status(moe::blk::launch_block_norm(a, static_cast<cudaStream_t>(stream)));
}

size_t moe_block_norm_workspace_size(int T, int H) {
  if (T < 0 || H <= 0 || H > kMaxNormH || T > kMaxT) return 0;
  return moe::blk::block_norm_ws_bytes(T, H);
}

moe_status moe_block_norm_backward(const void* dx_out, int64_t ld_dxo, const void* dn, int64_t ld_dn,
                                   const void* x_out, int64_t ldx_out, int x_type, const void* y, int64_t ldy,
                                   int y_type, const void* gate, int gate_kind, int64_t ld_gate,
                                   const float* gamma_post, const float* gamma_pre, int post_norm, float scale,
                                   const float* rstd_post, const float* rstd_pre, int T, int H, void* dx,
                                   int64_t ldx_grad, void* dy, int64_t ldy_grad, void* dgate, int64_t ld_dgate,
                                   float* dgamma_post, float* dgamma_pre, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  MOE_TRY(check_norm(x_type, y, y_type, gate, gate_kind, ld_gate, gamma_post, gamma_pre, post_norm, scale, T, H));
  moe::blk::NormGradArgs a{};
  const bool full = gate_kind == MOE_GATE_FULL;
  a.dx_out = rows(dx_out, ld_dxo, x_type);
  a.dn = rows(dn, ld_dn, y_type);
  a.x_out = rows(dn ? x_out : nullptr, ldx_out, x_type);
  a.y = rows(y, ldy, y_type);
  a.gate = rows(gate, full ? ld_gate : 0, y_type);
  a.dx = rows(dx, ldx_grad, x_type);
  a.dy = rows(dy, ldy_grad, y_type);
  a.dgate = rows(dgate, full ? ld_dgate : 0, y_type);
  MOE_TRY(check_rows(a.dx_out, T, H));
  MOE_TRY(check_rows(a.dn, T, H));
  MOE_TRY(check_rows(a.x_out, T, H));
  MOE_TRY(check_rows(a.y, T, H));
  MOE_TRY(check_rows(a.dx, T, H));
  MOE_TRY(check_rows(a.dy, T, H));
  if (full)
    MOE_TRY(check_rows(a.dgate, T, H));
  else if (!a4(dgate))
    return MOE_EINVAL;
  if (!a4(rstd_post) || !a4(rstd_pre) || !a4(dgamma_post) || !a4(dgamma_pre)) return MOE_EINVAL;
  if (dgate && gate_kind == MOE_GATE_NONE) return MOE_EINVAL;
  if (dgamma_post && !post_norm) return MOE_EINVAL;
  if (T > 0) {
    if ((!dx_out && !dn) || !dx || (y != nullptr) != (dy != nullptr)) return MOE_EINVAL;
    if (dn && (!x_out || !rstd_pre)) return MOE_EINVAL;
    if (!dn && (dgamma_pre || gamma_pre)) return MOE_EINVAL;
    if (post_norm && !rstd_post) return MOE_EINVAL;
    if ((dx == dx_out && ldx_grad != ld_dxo) || dx == dn || dx == x_out || dx == y || dx == dy) return MOE_EINVAL;
    if (dy && (dy == dn || dy == y || dy == dx_out || dy == x_out || dy == gate || dy == dgate)) return MOE_EINVAL;
  }
  if (dgate && dgate == gate) return MOE_EINVAL;
  if (dgamma_post || dgamma_pre || (dgate && gate_kind == MOE_GATE_CHANNEL)) {
    if (!workspace) return MOE_EWORKSPACE;
    if (!aligned(workspace, 16)) return MOE_EINVAL;
    if (workspace_bytes < moe_block_norm_workspace_size(T, H)) return MOE_EWORKSPACE;
  }
  a.gate_kind = gate_kind;
  a.post_norm = post_norm != 0;
  a.gamma_post = gamma_post;
  a.gamma_pre = gamma_pre;
  a.scale = scale;
  a.rstd_post = rstd_post;
  a.rstd_pre = rstd_pre;
  a.T = T;
  a.H = H;
  a.dgamma_post = dgamma_post;
  a.dgamma_pre = dgamma_pre;
  a.ws = static_cast<float*>(workspace);
  return cuda_status(moe::blk::launch_block_norm_grad(a, static_cast<cudaStream_t>(stream)));
}

size_t moe_route_backward_workspace_size(int T, int k, int E, int H) {
  if (T < 0 || k <= 0 || E <= 0 || H <= 0 || k > moe::kMaxK || E > moe::kMaxE || H > kMaxH || T > kMaxT ||
      static_cast<long long>(T) * k >= (1LL << 31))
    return 0;
  return moe::blk::route_grad_ws_bytes(T, k, E, H);
}

moe_status moe_route_backward(const float* dw, const float* topk_w, const int32_t* topk_ids, const uint16_t* x,
                              int64_t ldx, const uint16_t* w_router, int64_t ld_router, const int32_t* offsets,
                              const int32_t* perm, int T, int k, int E, int H, float* dlogits, void* dx,
                              int64_t ldx_grad, int dx_type, const void* add, int64_t ld_add, float* dw_router,
                              int64_t ld_dw, float* dbias, void* workspace, size_t workspace_bytes,
                              int32_t* dev_status, void* stream) {
  if (T < 0 || k <= 0 || E <= 0 || H <= 0) return MOE_ESHAPE;
  if (k > moe::kMaxK || k > E || E > moe::kMaxE || H > kMaxH || T > kMaxT) return MOE_ENOTSUP;
  if (static_cast<long long>(T) * k >= (1LL << 31)) return MOE_ENOTSUP;
  if (!type_ok(dx_type)) return MOE_EINVAL;
  moe::blk::RouteGradArgs a{};
  a.x = rows(x, ldx, MOE_ROW_BF16);
  a.w_router = rows(w_router, ld_router, MOE_ROW_BF16);
  a.dx = rows(dx, ldx_grad, dx_type);
  a.add = rows(dx ? add : nullptr, ld_add, dx_type);
  a.dw_router = rows(dw_router, ld_dw, MOE_ROW_F32);
  MOE_TRY(check_rows(a.x, T, H));
  MOE_TRY(check_rows(a.w_router, E, H));
  MOE_TRY(check_rows(a.dx, T, H));
  MOE_TRY(check_rows(a.add, T, H));
  MOE_TRY(check_rows(a.dw_router, E, H));
  if (!a4(dw) || !a4(topk_w) || !a4(topk_ids) || !a4(offsets) || !a4(perm) || !a4(dlogits) || !a4(dbias) ||
      !a4(dev_status))
    return MOE_EINVAL;
  if (T > 0) {
    if (!dw || !topk_w || !topk_ids || !dlogits) return MOE_EINVAL;
    if (dx && (!w_router || dx == w_router || dx == x || (add == dx && ld_add != ldx_grad))) return MOE_EINVAL;
    if (dw_router && !x) return MOE_EINVAL;
    if ((dw_router || dbias) && (!offsets || !perm)) return MOE_EINVAL;
    if (dlogits == dw || dlogits == topk_w) return MOE_EINVAL;
  }
  if (dw_router || dbias) {
    if (!workspace) return MOE_EWORKSPACE;
    if (!aligned(workspace, 16)) return MOE_EINVAL;
    if (workspace_bytes < moe_route_backward_workspace_size(T, k, E, H)) return MOE_EWORKSPACE;
  }
  a.dw = dw;
  a.w = topk_w;
  a.ids = topk_ids;
  a.offsets = offsets;
  a.perm = perm;
  a.T = T;
  a.k = k;
  a.E = E;
  a.H = H;
  a.dlogits = dlogits;
  a.dbias = dbias;
  a.ws = workspace;
  a.status = dev_status;
  return cuda_status(moe::blk::launch_route_grad(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
