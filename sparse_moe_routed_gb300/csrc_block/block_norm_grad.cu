// Gradient of the block norm (block_norm.cu).
//
// With xh = x_out r2, yh = y r1 (the normalised rows), u = dn c2, c1 = (1 +
// gamma_post) times a per-channel gate and g the gate where it varies by row:
//   D  = dx_out + r2 (u - xh mean(u xh)),   dx = scale D
//   q  = sum D c1 yh g  (per-token dgate: without g)
//   dy = r1 (D g c1 - yh q / H)
// Written with normalised rows, so that a small row's large r is never cubed.
// Per column, A = sum_t D g yh gives dgamma_post = gate_c A as well as a
// per-channel dgate = (1 + gamma_post) A, and B = sum_t dn xh is dgamma_pre:
// two accumulators per column, whatever the gate.
//
// Bound by HBM: four rows in, two out.  A group of threads owns a row, the
// rows ahead are staged in shared memory (stage.cuh) and read from there again
// in each of the row's three steps, which leaves the registers to D and the
// column sums.  One CTA per SM keeps A and B over all its rows and writes one
// partial row of each; a second launch adds these in order.
#include <math.h>

#include "norm.h"
#include "stage.cuh"

namespace moe {
namespace blk {

namespace {

constexpr int kThreads = 640;

template <typename TX, typename TY, int G, int NCH>
__global__ void __launch_bounds__(NCH == 1 ? kThreads : kMaxGroupThreads)
    block_norm_grad_kernel(const NormGradArgs a, const NormPlan p, int want_cols) {
  constexpr bool STAGED = NCH <= kMaxStagedChunks;
  constexpr int NA = STAGED ? NCH * 8 : 1;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float red[15][2][16];
  pdl_wait();
  pdl_trigger();
  const int nt = p.nt, H = a.H;
  const int group = threadIdx.x / nt, tid = threadIdx.x - group * nt;
  const bool has_d = a.dx_out.p != nullptr, has_n = a.dn.p != nullptr, has_y = a.y.p != nullptr;
  const bool full = a.gate_kind == MOE_GATE_FULL, token = a.gate_kind == MOE_GATE_TOKEN;
  const TX *dxo = static_cast<const TX*>(a.dx_out.p), *xo = static_cast<const TX*>(a.x_out.p);
  const TY *dn = static_cast<const TY*>(a.dn.p), *y = static_cast<const TY*>(a.y.p);
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
  // column sums: registers, or (unstaged, widest rows) the thread's own
  // places in shared memory
  float accA[NA], accB[NA];
#pragma unroll
  for (int i = 0; i < NA; ++i) accA[i] = accB[i] = 0.f;
  float* shA = reinterpret_cast<float*>(smem) + tid;
  float* shB = shA + NCH * 8 * nt;
  if (!STAGED)
    for (int i = 0; i < NCH * 8; ++i) shA[i * nt] = shB[i * nt] = 0.f;

  const int bx = NCH * nt * kSlot<TX>, by = NCH * nt * kSlot<TY>;
  const int off_x = has_d ? bx : 0, off_dn = off_x + (has_n ? bx : 0), off_y = off_dn + (has_n ? by : 0),
            off_g = off_y + (has_y ? by : 0);
  unsigned char* mine = smem + static_cast<size_t>(group) * p.stages * p.stage;
  const int64_t step = static_cast<int64_t>(gridDim.x) * p.groups;
  int64_t t = static_cast<int64_t>(blockIdx.x) * p.groups + group;
  auto stage = [&](int64_t row, int s) {
    if (row < a.T) {
      unsigned char* at = mine + static_cast<size_t>(s) * p.stage;
      if (has_n) {
        stage_row<TX, G, NCH>(at + off_x, xo + row * a.x_out.ld, tid, nt, H);
        stage_row<TY, G, NCH>(at + off_dn, dn + row * a.dn.ld, tid, nt, H);
      }
      if (has_d) stage_row<TX, G, NCH>(at, dxo + row * a.dx_out.ld, tid, nt, H);
      if (has_y) stage_row<TY, G, NCH>(at + off_y, y + row * a.y.ld, tid, nt, H);
      if (full) stage_row<TY, G, NCH>(at + off_g, gate + row * a.gate.ld, tid, nt, H);
    }
    copies_commit();
  };
  if (STAGED)
    for (int s = 0; s < p.stages - 1; ++s) stage(t + s * step, s);
  float r1n = 1.f, r2n = 0.f, gtn = 1.f;  // the next row's factors
  auto factors = [&](int64_t row) {
    if (row >= a.T) return;
    if (a.post_norm) r1n = a.rstd_post[row];
    if (has_n) r2n = a.rstd_pre[row];
    if (token) gtn = gate_v[row];
  };
  factors(t);
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
    const float r1 = r1n, r2 = r2n, gt = gtn;
    factors(t + step);
    auto read_x = [&](int off, const TX* q, int64_t ld, int h, float(&f)[8]) {
      if (STAGED)
        read_staged<TX, G>(at + off, h, tid, nt, f);
      else
        read_global<TX, G>(q + t * ld, h, tid, nt, H, f);
    };
    auto read_y = [&](int off, const TY* q, int64_t ld, int h, float(&f)[8]) {
      if (STAGED)
        read_staged<TY, G>(at + off, h, tid, nt, f);
      else
        read_global<TY, G>(q + t * ld, h, tid, nt, H, f);
    };
    auto c1_of = [&](int h, int i) {
      if (NCH == 1) return c1[NCH == 1 ? i : 0];
      const int c = col0<G>(h, i, tid, nt);
      return c < H ? c1_at(c) : 0.f;
    };
    auto c2_of = [&](int h, int i) {
      if (NCH == 1) return c2[NCH == 1 ? i : 0];
      const int c = col0<G>(h, i, tid, nt);
      return c < H ? gain(a.gamma_pre, c) : 0.f;
    };

    float m = 0.f;
    if (has_n) {
      float dot = 0.f;
#pragma unroll
      for (int h = 0; h < NCH; ++h) {
        float xv[8], dv[8];
        read_x(off_x, xo, a.x_out.ld, h, xv);
        read_y(off_dn, dn, a.dn.ld, h, dv);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float xh = xv[i] * r2;
          if (STAGED)
            accB[STAGED ? h * 8 + i : 0] = fmaf(dv[i], xh, accB[STAGED ? h * 8 + i : 0]);
          else
            shB[(h * 8 + i) * nt] = fmaf(dv[i], xh, shB[(h * 8 + i) * nt]);
          dot = fmaf(dv[i] * c2_of(h, i), xh, dot);
        }
      }
      m = group_sum(dot, red[group], which, tid, nt, group) * inv_h;
    }

    float D[NCH][8];
    float q = 0.f;
#pragma unroll
    for (int h = 0; h < NCH; ++h) {
      if (has_d) {
        read_x(0, dxo, a.dx_out.ld, h, D[h]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) D[h][i] = 0.f;
      }
      if (has_n) {
        float xv[8], dv[8];
        read_x(off_x, xo, a.x_out.ld, h, xv);
        read_y(off_dn, dn, a.dn.ld, h, dv);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          D[h][i] = fmaf(r2, fmaf(dv[i], c2_of(h, i), -(xv[i] * r2) * m), D[h][i]);
      }
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = a.scale * D[h][i];
      write_row<TX, G>(static_cast<TX*>(a.dx.p) + t * a.dx.ld, h, tid, nt, H, o);
      if (!has_y) continue;
      float yv[8], g[8];
      read_y(off_y, y, a.y.ld, h, yv);
      if (full) {
        read_y(off_g, gate, a.gate.ld, h, g);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = gt;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float yh = yv[i] * r1;
        const float dg = D[h][i] * g[i];
        if (STAGED)
          accA[STAGED ? h * 8 + i : 0] = fmaf(dg, yh, accA[STAGED ? h * 8 + i : 0]);
        else
          shA[(h * 8 + i) * nt] = fmaf(dg, yh, shA[(h * 8 + i) * nt]);
        const float c = c1_of(h, i);
        o[i] = D[h][i] * c * yh;  // a full gate's gradient
        D[h][i] = dg * c;
        q += token ? o[i] : D[h][i] * yh;
      }
      if (full && a.dgate.p != nullptr)
        write_row<TY, G>(static_cast<TY*>(a.dgate.p) + t * a.dgate.ld, h, tid, nt, H, o);
    }
    if (!has_y) continue;
    m = 0.f;
    if (a.post_norm || token) {
      q = group_sum(q, red[group], which, tid, nt, group);
      if (token) {
        if (tid == 0 && a.dgate.p != nullptr) static_cast<float*>(a.dgate.p)[t] = q;
        q *= gt;
      }
      m = q * inv_h;
    }
#pragma unroll
    for (int h = 0; h < NCH; ++h) {
      if (a.post_norm) {
        float yv[8];
        read_y(off_y, y, a.y.ld, h, yv);
#pragma unroll
        for (int i = 0; i < 8; ++i) D[h][i] = r1 * fmaf(-(yv[i] * r1), m, D[h][i]);
      }
      write_row<TY, G>(static_cast<TY*>(a.dy.p) + t * a.dy.ld, h, tid, nt, H, D[h]);
    }
  }
  if (!want_cols) return;
  // the groups' sums, added in group order, then one partial row of A and B
  if (STAGED && p.groups > 1) {
    float* sh = reinterpret_cast<float*>(smem);
    __syncthreads();
    if (group > 0) {
      float* s = sh + static_cast<size_t>(group - 1) * 2 * NA * nt + tid;
#pragma unroll
      for (int i = 0; i < NA; ++i) {
        s[i * nt] = accA[i];
        s[(NA + i) * nt] = accB[i];
      }
    }
    __syncthreads();
    if (group > 0) return;
    for (int k = 0; k + 1 < p.groups; ++k) {
      const float* s = sh + static_cast<size_t>(k) * 2 * NA * nt + tid;
#pragma unroll
      for (int i = 0; i < NA; ++i) {
        accA[i] += s[i * nt];
        accB[i] += s[(NA + i) * nt];
      }
    }
  }
  float* w = a.ws + static_cast<size_t>(blockIdx.x) * 2 * H;
#pragma unroll
  for (int h = 0; h < NCH; ++h)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = col0<G>(h, i, tid, nt);
      if (c >= H) continue;
      w[c] = STAGED ? accA[STAGED ? h * 8 + i : 0] : shA[(h * 8 + i) * nt];
      w[H + c] = STAGED ? accB[STAGED ? h * 8 + i : 0] : shB[(h * 8 + i) * nt];
    }
}

// Column sums over the parts, in part order within each of the CTA's 8 rows
// of threads, then over those.
__global__ void __launch_bounds__(256) norm_cols_kernel(const float* __restrict__ ws, int parts, int H,
                                                        const float* gate_c, const float* gamma_post, int post_norm,
                                                        float* dgate_c, float* dgamma_post, float* dgamma_pre) {
  __shared__ float sh[2][8][32];
  pdl_wait();
  pdl_trigger();
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + tx;
  float A = 0.f, B = 0.f;
  if (col < H) {
#pragma unroll 4
    for (int p = ty; p < parts; p += 8) {
      const float* w = ws + static_cast<size_t>(p) * 2 * H;
      A += w[col];
      B += w[H + col];
    }
  }
  sh[0][ty][tx] = A;
  sh[1][ty][tx] = B;
  __syncthreads();
  if (ty != 0 || col >= H) return;
  A = B = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    A += sh[0][i][tx];
    B += sh[1][i][tx];
  }
  if (dgamma_post != nullptr) dgamma_post[col] = gate_c != nullptr ? gate_c[col] * A : A;
  if (dgate_c != nullptr) dgate_c[col] = post_norm ? gain(gamma_post, col) * A : A;
  if (dgamma_pre != nullptr) dgamma_pre[col] = B;
}

}  // namespace

// One partial row of A and B per CTA, at most one CTA per SM and token.
size_t block_norm_ws_bytes(int T, int H) {
  const size_t parts = std::max(1, std::min(T, sm_count()));
  return (parts * 2 * H * sizeof(float) + 255) / 256 * 256;
}

cudaError_t launch_block_norm_grad(const NormGradArgs& a, cudaStream_t st) {
  const bool chan = a.gate_kind == MOE_GATE_CHANNEL;
  float* dgate_c = chan ? static_cast<float*>(a.dgate.p) : nullptr;
  const int want = a.dgamma_post != nullptr || a.dgamma_pre != nullptr || dgate_c != nullptr;
  int parts = 0;
  if (a.T > 0) {
    const bool full = a.gate_kind == MOE_GATE_FULL;
    const Rows none = {nullptr, 0, MOE_ROW_F32};
    const Rows gate = full ? a.gate : none, dgate = full ? a.dgate : none;
    const int slot = row_bytes8(a.dx_out) + row_bytes8(a.x_out) + row_bytes8(a.dn) + row_bytes8(a.y) + row_bytes8(gate);
    NormPlan p = norm_plan(a.T, a.H, slot, kThreads);
    p.grid = std::min(p.grid, sm_count());
    const int cols = p.nch <= kMaxStagedChunks ? (p.groups - 1) * 2 * p.nch * 8 * p.nt * 4 : 2 * p.nch * 8 * p.nt * 4;
    p.smem = std::max(p.smem, cols);
    parts = p.grid;
    const int unit = norm_unit({a.dx_out, a.x_out, a.dn, a.y, gate, dgate, a.dx, a.dy});
    const cudaError_t e = norm_dispatch(a.dx.type, a.y.type, unit, p.nch, [&](auto tx, auto ty, auto g, auto n) {
      auto kern = block_norm_grad_kernel<decltype(tx), decltype(ty), decltype(g)::value, decltype(n)::value>;
      static std::atomic<uint64_t> done{0};
      const cudaError_t r = allow_smem(kern, done);
      if (r != cudaSuccess) return r;
      return launch_pdl(kern, dim3(p.grid), dim3(p.nt * p.groups), p.smem, st, a, p, want);
    });
    if (e != cudaSuccess) return e;
  }
  if (!want) return cudaSuccess;
  return launch_pdl(norm_cols_kernel, dim3((a.H + 31) / 32), dim3(256), 0, st, a.ws, parts, a.H,
                    chan ? static_cast<const float*>(a.gate.p) : nullptr, a.gamma_post, a.post_norm, dgate_c,
                    a.dgamma_post, a.dgamma_pre);
}

}  // namespace blk
}  // namespace moe
