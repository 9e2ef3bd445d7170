// Internal launchers of libmoe_block (host side).  Each returns the CUDA
// error of its launches; the extern "C" layer in api.cu validates arguments
// first.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

#include "../../include/moe_block.h"

namespace moe {
namespace blk {

// Multiprocessors of the current device, at least 1.
int sm_count();

// Launch with programmatic stream serialization (see pdl_wait in
// ../csrc/common.cuh): every kernel waits before its first global access and
// before its trigger.  (The later launches of an ffn.cu call read offsets and
// weights before: the launch before them triggered after its wait.)  libmoe's int4 contractions may read offsets and packed
// records while a launch of this library right before them still runs (see the
// stream token in ../csrc/launch.h): no kernel that triggers writes those.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                       Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<Args&&>(args)...);
}

// A matrix of rows: element (i, c) is at p[i * ld + c], of type moe_row_type.
struct Rows {
  void* p;
  int64_t ld;
  int type;
};

// Rows that start on u-element boundaries (null rows do).
inline bool starts_on(const Rows& r, int u) {
  return r.p == nullptr ||
         (r.ld % u == 0 && reinterpret_cast<uintptr_t>(r.p) % (u * (r.type == MOE_ROW_F32 ? 4 : 2)) == 0);
}
// The unit (rows.cuh) that all of these rows allow: 8, 2 or 1.
inline int row_unit(std::initializer_list<Rows> all) {
  int u = 8;
  for (const Rows& r : all) {
    if (u == 8 && !starts_on(r, 8)) u = 2;
    if (u == 2 && !starts_on(r, 2)) u = 1;
  }
  return u;
}

// dispatch.cu.  slot_of [T,k]; weights or NULL.
// out[slot] = w * tok[t];  with dw, dw[t,j] = <tok[t], dot[slot]>
cudaError_t launch_spread(const Rows& tok, const Rows& dot, const int32_t* slot_of, const float* w, int T, int k,
                          int H, int R, const Rows& out, float* dw, int32_t* status, cudaStream_t st);
// out[t] = add[t] + sum_j w * rows[slot];  with dw, dw[t,j] = <rows[slot], dot[t]>
cudaError_t launch_join(const Rows& rows, const Rows& dot, const int32_t* slot_of, const float* w, int T, int k,
                        int H, int R, const Rows& out, const Rows& add, float* dw, int32_t* status, cudaStream_t st);

// block_norm.cu
struct NormArgs {
  Rows x, y, gate, x_out, n_out;
  int gate_kind, post_norm;
  const float *gamma_post, *gamma_pre;
  float scale, eps;
  int T, H;
  float *rstd_post, *rstd_pre;
};
cudaError_t launch_block_norm(const NormArgs& a, cudaStream_t st);

struct NormGradArgs {
  Rows dx_out, dn, x_out, y, gate, dx, dy, dgate;
  int gate_kind, post_norm;
  const float *gamma_post, *gamma_pre;
  float scale;
  const float *rstd_post, *rstd_pre;
  int T, H;
  float *dgamma_post, *dgamma_pre;
  float* ws;
};
size_t block_norm_ws_bytes(int T, int H);
cudaError_t launch_block_norm_grad(const NormGradArgs& a, cudaStream_t st);

// route_grad.cu
struct RouteGradArgs {
  const float *dw, *w;
  const int32_t* ids;
  Rows x, w_router;
  const int32_t *offsets, *perm;
  int T, k, E, H;
  float* dlogits;
  Rows dx, add, dw_router;
  float* dbias;
  void* ws;
  int32_t* status;
};
size_t route_grad_ws_bytes(int T, int k, int E, int H);
cudaError_t launch_route_grad(const RouteGradArgs& a, cudaStream_t st);

// checkpoint.cu.  q [T,H] int8, exp [T, ceil(H/32)]: rows of bytes.
struct Bytes {
  uint8_t* p;
  int64_t ld;
};
cudaError_t launch_checkpoint_save(const Rows& x, int T, int H, const Bytes& q, const Bytes& exp, cudaStream_t st);
// slot_of NULL: out [T,H]
cudaError_t launch_checkpoint_load(const Bytes& q, const Bytes& exp, int T, int H, const int32_t* slot_of,
                                   const float* w, int k, int R, const Rows& out, int32_t* status, cudaStream_t st);

// ffn.cu
struct Act {
  void* p;
  int kind;
  int64_t ld;
  Bytes exp;
};
struct FfnArgs {
  Rows x;
  const uint16_t *w_gateup, *w_down;
  const int32_t* offsets;
  int R, E, H, I;
  uint16_t* h;  // [R,I]
  Act act;
  Rows y;
  int32_t* status;
};
cudaError_t launch_ffn(const FfnArgs& a, cudaStream_t st);

struct FfnGradArgs {
  Rows dy, x;
  const uint16_t *w_gateup, *w_down;
  const int32_t* offsets;
  int R, E, H, I;
  Act act;
  Rows dx;
  void *dw_gateup, *dw_down;
  int dw_type, accumulate;
  uint16_t *da, *h;  // workspace: [R,2I], [R,I],
  int* queue;        // a word
  int32_t* status;
};
cudaError_t launch_ffn_grad(const FfnGradArgs& a, cudaStream_t st);

}  // namespace blk
}  // namespace moe
