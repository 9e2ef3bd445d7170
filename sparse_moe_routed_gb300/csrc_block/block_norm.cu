// The norms on both sides of a block with its gate and the residual scale, in
// one pass over the rows.
//
// AFN-001 "Porting Qwen3.8-Flash-Next to Hebrus", section "Phase 1: separate
// math from acceleration": zero-centred RMS normalisation (gain 1 + gamma).
//
// Per row, with c1 = (1 + gamma_post) times a per-channel gate, c2 = 1 +
// gamma_pre and g the gate where it varies by row:
//   x_out = scale x + g c1 y r1,   n = x_out r2 c2
//
// Bound by HBM: every operand's row moves once.  A group of threads owns a
// row; the rows ahead are staged in shared memory (stage.cuh), c1 and c2 stay
// in registers for the launch.
#include <math.h>

#include "norm.h"
#include "stage.cuh"

namespace moe {
namespace blk {

namespace {

constexpr int kThreads = 1024;

template <typename TX, typename TY, int G, int NCH>
__global__ void __launch_bounds__(NCH == 1 ? kThreads : kMaxGroupThreads)
    block_norm_kernel(const NormArgs a, const NormPlan p) {
  constexpr bool STAGED = NCH <= kMaxStagedChunks;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float red[15][2][16];
  pdl_wait();
  pdl_trigger();
  const int nt = p.nt, H = a.H;
  const int group = threadIdx.x / nt, tid = threadIdx.x - group * nt;
  const bool has_y = a.y.p != nullptr, has_n = a.n_out.p != nullptr;
  const bool full = a.gate_kind == MOE_GATE_FULL, token = a.gate_kind == MOE_GATE_TOKEN;
  const TX* x = static_cast<const TX*>(a.x.p);
  const TY* y = static_cast<const TY*>(a.y.p);
  const TY* gate = static_cast<const TY*>(a.gate.p);
  const float* gate_v = static_cast<const float*>(a.gate.p);
  const float inv_h = 1.0f / static_cast<float>(H);
  auto c1_at = [&](int c) {
    float v = a.post_norm ? gain(a.gamma_post, c) : 1.0f;
    if (a.gate_kind == MOE_GATE_CHANNEL) v *= gate_v[c];
    return v;
  };
  float c1[NCH == 1 ? 8 : 1], c2[NCH == 1 ? 8 : 1];
  if (NCH == 1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = col0<G>(0, i, tid, nt);
      c1[NCH == 1 ? i : 0] = has_y && c < H ? c1_at(c) : 0.f;
      c2[NCH == 1 ? i : 0] = c < H ? gain(a.gamma_pre, c) : 0.f;
    }
  }
  const int off_y = NCH * nt * kSlot<TX>, off_g = off_y + (has_y ? NCH * nt * kSlot<TY> : 0);
  unsigned char* mine = smem + static_cast<size_t>(group) * p.stages * p.stage;
  const int64_t step = static_cast<int64_t>(gridDim.x) * p.groups;
  int64_t t = static_cast<int64_t>(blockIdx.x) * p.groups + group;
  auto stage = [&](int64_t row, int s) {
    if (row < a.T) {
      unsigned char* at = mine + static_cast<size_t>(s) * p.stage;
      stage_row<TX, G, NCH>(at, x + row * a.x.ld, tid, nt, H);
      if (has_y) stage_row<TY, G, NCH>(at + off_y, y + row * a.y.ld, tid, nt, H);
      if (full) stage_row<TY, G, NCH>(at + off_g, gate + row * a.gate.ld, tid, nt, H);
    }
    copies_commit();
  };
  if (STAGED)
    for (int s = 0; s < p.stages - 1; ++s) stage(t + s * step, s);
  float gt_next = token && t < a.T ? gate_v[t] : 1.0f;
  int which = 0, slot = 0;
  for (; t < a.T; t += step) {
    const unsigned char* at = mine + static_cast<size_t>(slot) * p.stage;
    if (STAGED) {
      if (p.stages == 1) {
        stage(t, 0);
        copies_wait(0);
      } else {
        copies_wait(p.stages - 2);
        stage(t + (p.stages - 1) * step, slot == 0 ? p.stages - 1 : slot - 1);
      }
      slot = slot + 1 == p.stages ? 0 : slot + 1;
    }
    const float gt = gt_next;
    if (token && t + step < a.T) gt_next = gate_v[t + step];
    auto read_y = [&](int h, float(&f)[8]) {
      if (STAGED)
        read_staged<TY, G>(at + off_y, h, tid, nt, f);
      else
        read_global<TY, G>(y + t * a.y.ld, h, tid, nt, H, f);
    };
    float r1 = gt;  // the factor of c1 y: the norm's and the token's
    if (has_y && a.post_norm) {
      float ss = 0.f;
#pragma unroll
      for (int h = 0; h < NCH; ++h) {
        float f[8];
        read_y(h, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
      }
      r1 = 1.0f / sqrtf(group_sum(ss, red[group], which, tid, nt, group) * inv_h + a.eps);
      if (tid == 0 && a.rstd_post != nullptr) a.rstd_post[t] = r1;
    }
    float xo[NCH][8];
    float ss = 0.f;
#pragma unroll
    for (int h = 0; h < NCH; ++h) {
      if (STAGED)
        read_staged<TX, G>(at, h, tid, nt, xo[h]);
      else
        read_global<TX, G>(x + t * a.x.ld, h, tid, nt, H, xo[h]);
#pragma unroll
      for (int i = 0; i < 8; ++i) xo[h][i] *= a.scale;
      if (has_y) {
        float f[8];
        read_y(h, f);
        // y r1 first: the normalised value, which neither factor can overflow
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= r1;
        if (a.post_norm && token) {
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] *= gt;
        }
        if (full) {
          float g[8];
          if (STAGED)
            read_staged<TY, G>(at + off_g, h, tid, nt, g);
          else
            read_global<TY, G>(gate + t * a.gate.ld, h, tid, nt, H, g);
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] *= g[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float c = c1[NCH == 1 ? i : 0];
          if (NCH > 1) {
            const int col = col0<G>(h, i, tid, nt);
            c = col < H ? c1_at(col) : 0.f;
          }
          xo[h][i] = fmaf(f[i], c, xo[h][i]);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(xo[h][i], xo[h][i], ss);
      if (a.x_out.p != nullptr)
        write_row<TX, G>(static_cast<TX*>(a.x_out.p) + t * a.x_out.ld, h, tid, nt, H, xo[h]);
    }
    if (!has_n) continue;
    const float r2 = 1.0f / sqrtf(group_sum(ss, red[group], which, tid, nt, group) * inv_h + a.eps);
    if (tid == 0 && a.rstd_pre != nullptr) a.rstd_pre[t] = r2;
#pragma unroll
    for (int h = 0; h < NCH; ++h) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float c = c2[NCH == 1 ? i : 0];
        if (NCH > 1) {
          const int col = col0<G>(h, i, tid, nt);
          c = col < H ? gain(a.gamma_pre, col) : 0.f;
        }
        xo[h][i] = xo[h][i] * r2 * c;
      }
      write_row<TY, G>(static_cast<TY*>(a.n_out.p) + t * a.n_out.ld, h, tid, nt, H, xo[h]);
    }
  }
}

}  // namespace

cudaError_t launch_block_norm(const NormArgs& a, cudaStream_t st) {
  const bool full = a.gate_kind == MOE_GATE_FULL;
  const Rows gate = full ? a.gate : Rows{nullptr, 0, MOE_ROW_F32};
  const NormPlan p = norm_plan(a.T, a.H, row_bytes8(a.x) + row_bytes8(a.y) + row_bytes8(gate), kThreads);
  const int unit = norm_unit({a.x, a.y, gate, a.x_out, a.n_out});
  return norm_dispatch(a.x.type, a.y.type, unit, p.nch, [&](auto tx, auto ty, auto g, auto n) {
    auto kern = block_norm_kernel<decltype(tx), decltype(ty), decltype(g)::value, decltype(n)::value>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(kern, done);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(p.grid), dim3(p.nt * p.groups), p.smem, st, a, p);
  });
}

}  // namespace blk
}  // namespace moe
