// The norms on both sides of a block with its gate and the residual scale in
// one pass over the rows, and their gradient.
//
// AFN-001 "Porting Qwen3.8-Flash-Next to Hebrus", section "Phase 1: separate
// math from acceleration": zero-centred RMS normalisation (gain 1 + gamma).
//
// Forward, per row (yh = y r1 is the normalised block output):
//   x_out = scale x + c1 yh g,   n = x_out r2 c2
// with c1 = (1 + gamma_post) times a per-channel gate, c2 = 1 + gamma_pre and
// g the gate where it varies by row.  Gradient, with xh = x_out r2 and
// u = dn c2 (two reductions per row, each over products of normalised values,
// so that a small row's large r cannot overflow r^3):
//   D  = dx_out + r2 (u - xh mean(u xh))
//   q  = sum D c1 yh
//   dy = r1 (D g c1 - yh g q / H),   dx = scale D,   per-token dgate = q
// Per column, A = sum_t D g yh gives both dgamma_post = gate_c A and a
// per-channel dgate = (1 + gamma_post) A, and B = sum_t dn xh is dgamma_pre.
//
// Bound by HBM: each row of each operand moves once; a row lives in the
// registers of one group of threads (eight elements a thread and chunk)
// between its reads and its writes.
#include <math.h>

#include <algorithm>

#include "launch.h"
#include "rows.cuh"

namespace moe {
namespace blk {

namespace {

constexpr int kMaxThreads = 512;  // threads of a group, at 8 * NCH elements each
constexpr int kMaxParts = 1024;   // partial column sums of the gradient

// How a launch cuts rows: groups of `nt` threads, `rp` groups per CTA.
struct Shape {
  int nt, rp, nch, grid;
};

Shape shape_for(int T, int H) {
  Shape s;
  const int chunks = (H + 7) / 8;
  s.nch = chunks <= kMaxThreads ? 1 : chunks <= 2 * kMaxThreads ? 2 : 4;
  s.nt = ((chunks + s.nch - 1) / s.nch + 31) / 32 * 32;
  s.rp = std::max(1, std::min(4, 256 / s.nt));
  const int per_sm = std::max(1, 1024 / (s.nt * s.rp));
  s.grid = std::min((T + s.rp - 1) / s.rp, sm_count() * per_sm);
  s.grid = std::max(1, std::min(s.grid, kMaxParts / s.rp));
  return s;
}

// Sum of v over the group's nt threads; alternate `buf` between successive
// sums: a buffer is written again only after the barrier of the sum between.
__device__ __forceinline__ float group_sum(float v, float (*buf)[kMaxThreads / 32], int& which, int tid, int nt,
                                           int group) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (nt == 32) return v;
  float* b = buf[which];
  which ^= 1;
  if ((tid & 31) == 0) b[tid >> 5] = v;
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(nt) : "memory");
  float s = 0.f;
  for (int i = 0; i < nt / 32; ++i) s += b[i];
  return s;
}

// c1 and c2 of a thread's columns.
__device__ __forceinline__ float gain(const float* gamma, int c) { return gamma != nullptr ? 1.0f + gamma[c] : 1.0f; }

template <typename TX, typename TY, bool VEC, int NCH>
__global__ void __launch_bounds__(kMaxThreads) block_norm_kernel(const NormArgs a, int nt) {
  __shared__ float red[8][2][kMaxThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int group = threadIdx.x / nt, tid = threadIdx.x - group * nt;
  const int groups = blockDim.x / nt;
  const int H = a.H;
  const bool has_y = a.y.p != nullptr, has_n = a.n_out.p != nullptr;
  const TX* x = static_cast<const TX*>(a.x.p);
  const TY* y = static_cast<const TY*>(a.y.p);
  const float* gate_v = static_cast<const float*>(a.gate.p);
  const float inv_h = 1.0f / static_cast<float>(H);
  int which = 0;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * groups + group; t < a.T;
       t += static_cast<int64_t>(gridDim.x) * groups) {
    float xo[NCH][8], yv[NCH][8];
    float ss = 0.f;
#pragma unroll
    for (int h = 0; h < NCH; ++h) {
      const Cols<VEC> c(h * nt * 8, tid, nt);
      Raw8<TX> xr;
      load8<VEC>(x + t * a.x.ld, c, H, xr);
      unpack(xr, xo[h]);
      if (has_y) {
        Raw8<TY> yr;
        load8<VEC>(y + t * a.y.ld, c, H, yr);
        unpack(yr, yv[h]);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(yv[h][i], yv[h][i], ss);
      }
    }
    float r1 = 1.0f;
    if (a.post_norm) {
      r1 = 1.0f / sqrtf(group_sum(ss, red[group], which, tid, nt, group) * inv_h + a.eps);
      if (tid == 0 && a.rstd_post != nullptr) a.rstd_post[t] = r1;
    }
    const float gt = a.gate_kind == MOE_GATE_TOKEN ? gate_v[t] : 1.0f;
    ss = 0.f;
#pragma unroll
    for (int h = 0; h < NCH; ++h) {
      const Cols<VEC> c(h * nt * 8, tid, nt);
      float gf[8];
      if (a.gate_kind == MOE_GATE_FULL) {
        Raw8<TY> gr;
        load8<VEC>(static_cast<const TY*>(a.gate.p) + t * a.gate.ld, c, H, gr);
        unpack(gr, gf);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int col = c.first + i * c.step;
        if (col >= H) continue;
        float v = a.scale * xo[h][i];
        if (has_y) {
          float z = yv[h][i] * r1 * gt;
          if (a.post_norm) z *= gain(a.gamma_post, col);
          if (a.gate_kind == MOE_GATE_CHANNEL) z *= gate_v[col];
          if (a.gate_kind == MOE_GATE_FULL) z *= gf[i];
          v += z;
        }
        xo[h][i] = v;
        ss = fmaf(v, v, ss);
      }
      if (a.x_out.p != nullptr) store8<VEC>(static_cast<TX*>(a.x_out.p) + t * a.x_out.ld, c, H, xo[h]);
    }
    if (has_n) {
      const float r2 = 1.0f / sqrtf(group_sum(ss, red[group], which, tid, nt, group) * inv_h + a.eps);
      if (tid == 0 && a.rstd_pre != nullptr) a.rstd_pre[t] = r2;
#pragma unroll
      for (int h = 0; h < NCH; ++h) {
        const Cols<VEC> c(h * nt * 8, tid, nt);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int col = c.first + i * c.step;
          if (col < H) xo[h][i] *= r2 * gain(a.gamma_pre, col);
        }
        store8<VEC>(static_cast<TY*>(a.n_out.p) + t * a.n_out.ld, c, H, xo[h]);
      }
    }
  }
}

// ws: [parts][2][H] column sums A and B, one part per group.
template <typename TX, typename TY, bool VEC, int NCH>
__global__ void __launch_bounds__(kMaxThreads) block_norm_grad_kernel(const NormGradArgs a, int nt, int want_cols) {
  __shared__ float red[8][2][kMaxThreads / 32];
  extern __shared__ float cols_sh[];  // NCH > 1: A and B, [2][NCH * nt * 8], each thread its own columns
  pdl_wait();
  pdl_trigger();
  const int group = threadIdx.x / nt, tid = threadIdx.x - group * nt;
  const int groups = blockDim.x / nt;
  const int H = a.H;
  const bool has_y = a.y.p != nullptr, has_n = a.dn.p != nullptr;
  const float* gate_v = static_cast<const float*>(a.gate.p);
  const float inv_h = 1.0f / static_cast<float>(H);
  float accA[NCH == 1 ? 8 : 1], accB[NCH == 1 ? 8 : 1];
  float* shA = cols_sh + tid * 8;
  float* shB = shA + NCH * nt * 8;
#pragma unroll
  for (int i = 0; i < (NCH == 1 ? 8 : 1); ++i) accA[i] = accB[i] = 0.f;
  if (NCH > 1) {
    for (int h = 0; h < NCH; ++h)
      for (int i = 0; i < 8; ++i) shA[h * nt * 8 + i] = shB[h * nt * 8 + i] = 0.f;
  }
  int which = 0;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * groups + group; t < a.T;
       t += static_cast<int64_t>(gridDim.x) * groups) {
    const float r2 = has_n ? a.rstd_pre[t] : 0.f;
    const float r1 = a.post_norm ? a.rstd_post[t] : 1.f;
    const float gt = a.gate_kind == MOE_GATE_TOKEN ? gate_v[t] : 1.0f;
    float D[NCH][8], xh[NCH][8], u[NCH][8];
    float dot = 0.f;
#pragma unroll
    for (int h = 0; h < NCH; ++h) {
      const Cols<VEC> c(h * nt * 8, tid, nt);
      if (a.dx_out.p != nullptr) {
        Raw8<TX> r;
        load8<VEC>(static_cast<const TX*>(a.dx_out.p) + t * a.dx_out.ld, c, H, r);
        unpack(r, D[h]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) D[h][i] = 0.f;
      }
      if (has_n) {
        Raw8<TX> r;
        load8<VEC>(static_cast<const TX*>(a.x_out.p) + t * a.x_out.ld, c, H, r);
        unpack(r, xh[h]);
        Raw8<TY> d;
        load8<VEC>(static_cast<const TY*>(a.dn.p) + t * a.dn.ld, c, H, d);
        unpack(d, u[h]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int col = c.first + i * c.step;
          if (col >= H) continue;
          xh[h][i] *= r2;
          if (NCH == 1)
            accB[NCH == 1 ? i : 0] = fmaf(u[h][i], xh[h][i], accB[NCH == 1 ? i : 0]);
          else
            shB[h * nt * 8 + i] = fmaf(u[h][i], xh[h][i], shB[h * nt * 8 + i]);
          u[h][i] *= gain(a.gamma_pre, col);
          dot = fmaf(u[h][i], xh[h][i], dot);
        }
      }
    }
    if (has_n) {
      const float m = group_sum(dot, red[group], which, tid, nt, group) * inv_h;
#pragma unroll
      for (int h = 0; h < NCH; ++h)
#pragma unroll
        for (int i = 0; i < 8; ++i) D[h][i] = fmaf(r2, u[h][i] - xh[h][i] * m, D[h][i]);
    }
    // the normalised block output takes xh's place, D g c1 takes u's
    float q = 0.f;
#pragma unroll
    for (int h = 0; h < NCH; ++h) {
      const Cols<VEC> c(h * nt * 8, tid, nt);
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = a.scale * D[h][i];
      store8<VEC>(static_cast<TX*>(a.dx.p) + t * a.dx.ld, c, H, o);
      if (!has_y) continue;
      Raw8<TY> r;
      load8<VEC>(static_cast<const TY*>(a.y.p) + t * a.y.ld, c, H, r);
      unpack(r, xh[h]);
      float gf[8];
      if (a.gate_kind == MOE_GATE_FULL) {
        Raw8<TY> gr;
        load8<VEC>(static_cast<const TY*>(a.gate.p) + t * a.gate.ld, c, H, gr);
        unpack(gr, gf);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) gf[i] = gt;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int col = c.first + i * c.step;
        if (col >= H) continue;
        float c1 = a.post_norm ? gain(a.gamma_post, col) : 1.0f;
        if (a.gate_kind == MOE_GATE_CHANNEL) c1 *= gate_v[col];
        xh[h][i] *= r1;
        const float dg = D[h][i] * gf[i];
        if (NCH == 1)
          accA[NCH == 1 ? i : 0] = fmaf(dg, xh[h][i], accA[NCH == 1 ? i : 0]);
        else
          shA[h * nt * 8 + i] = fmaf(dg, xh[h][i], shA[h * nt * 8 + i]);
        u[h][i] = dg * c1;
        const float dz = D[h][i] * c1 * xh[h][i];  // full gate: its gradient
        o[i] = dz;
        q = fmaf(a.gate_kind == MOE_GATE_TOKEN ? D[h][i] * c1 : u[h][i], xh[h][i], q);
      }
      if (a.gate_kind == MOE_GATE_FULL && a.dgate.p != nullptr)
        store8<VEC>(static_cast<TY*>(a.dgate.p) + t * a.dgate.ld, c, H, o);
    }
    if (!has_y) continue;
    float m = 0.f;
    if (a.post_norm || a.gate_kind == MOE_GATE_TOKEN) {
      q = group_sum(q, red[group], which, tid, nt, group);
      if (a.gate_kind == MOE_GATE_TOKEN) {
        if (tid == 0 && a.dgate.p != nullptr) static_cast<float*>(a.dgate.p)[t] = q;
        q *= gt;
      }
      m = a.post_norm ? q * inv_h : 0.f;
    }
#pragma unroll
    for (int h = 0; h < NCH; ++h) {
      const Cols<VEC> c(h * nt * 8, tid, nt);
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = a.post_norm ? r1 * (u[h][i] - xh[h][i] * m) : u[h][i];
      store8<VEC>(static_cast<TY*>(a.dy.p) + t * a.dy.ld, c, H, o);
    }
  }
  if (want_cols) {
    float* w = a.ws + (static_cast<size_t>(blockIdx.x) * groups + group) * 2 * H;
#pragma unroll
    for (int h = 0; h < NCH; ++h) {
      const Cols<VEC> c(h * nt * 8, tid, nt);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int col = c.first + i * c.step;
        if (col >= H) continue;
        w[col] = NCH == 1 ? accA[NCH == 1 ? i : 0] : shA[h * nt * 8 + i];
        w[H + col] = NCH == 1 ? accB[NCH == 1 ? i : 0] : shB[h * nt * 8 + i];
      }
    }
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

// f(type tag of x, type tag of y, vector flag)
template <typename F>
cudaError_t by_types(int xt, int yt, bool vec, F&& f) {
  auto g = [&](auto tx, auto ty) {
    return vec ? f(tx, ty, std::true_type()) : f(tx, ty, std::false_type());
  };
  if (xt == MOE_ROW_F32) return yt == MOE_ROW_F32 ? g(float(), float()) : g(float(), bf16_t());
  return yt == MOE_ROW_F32 ? g(bf16_t(), float()) : g(bf16_t(), bf16_t());
}

}  // namespace

cudaError_t launch_block_norm(const NormArgs& a, cudaStream_t st) {
  const Shape s = shape_for(a.T, a.H);
  const bool vec = vec_ok(a.x) && vec_ok(a.y) && vec_ok(a.x_out) && vec_ok(a.n_out) &&
                   (a.gate_kind != MOE_GATE_FULL || vec_ok(a.gate));
  return by_types(a.x.type, a.y.type, vec, [&](auto tx, auto ty, auto v) {
    using TX = decltype(tx);
    using TY = decltype(ty);
    constexpr bool V = decltype(v)::value;
    const dim3 g(s.grid), b(s.nt * s.rp);
    if (s.nch == 1) return launch_pdl(block_norm_kernel<TX, TY, V, 1>, g, b, 0, st, a, s.nt);
    if (s.nch == 2) return launch_pdl(block_norm_kernel<TX, TY, V, 2>, g, b, 0, st, a, s.nt);
    return launch_pdl(block_norm_kernel<TX, TY, V, 4>, g, b, 0, st, a, s.nt);
  });
}

size_t block_norm_ws_bytes(int T, int H) {
  const Shape s = shape_for(std::max(T, 1), H);
  return (static_cast<size_t>(s.grid) * s.rp * 2 * H * sizeof(float) + 255) / 256 * 256;
}

cudaError_t launch_block_norm_grad(const NormGradArgs& a, cudaStream_t st) {
  const Shape s = shape_for(std::max(a.T, 1), a.H);
  const bool chan = a.gate_kind == MOE_GATE_CHANNEL;
  float* dgate_c = chan ? static_cast<float*>(a.dgate.p) : nullptr;
  const int want = a.dgamma_post != nullptr || a.dgamma_pre != nullptr || dgate_c != nullptr;
  if (a.T > 0) {
    const bool full = a.gate_kind == MOE_GATE_FULL;
    const bool vec = vec_ok(a.dx_out) && vec_ok(a.dn) && vec_ok(a.x_out) && vec_ok(a.y) && vec_ok(a.dx) &&
                     vec_ok(a.dy) && (!full || (vec_ok(a.gate) && vec_ok(a.dgate)));
    const cudaError_t e = by_types(a.dx.type, a.y.type, vec, [&](auto tx, auto ty, auto v) {
      using TX = decltype(tx);
      using TY = decltype(ty);
      constexpr bool V = decltype(v)::value;
      const dim3 g(s.grid), b(s.nt * s.rp);
      auto go = [&](auto kern, size_t smem) {
        if (smem > 48 * 1024) {
          const cudaError_t r = cudaFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                                     cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                     static_cast<int>(smem));
          if (r != cudaSuccess) return r;
        }
        return launch_pdl(kern, g, b, smem, st, a, s.nt, want);
      };
      const size_t smem = static_cast<size_t>(2) * s.nch * s.nt * 8 * sizeof(float);
      if (s.nch == 1) return go(block_norm_grad_kernel<TX, TY, V, 1>, 0);
      if (s.nch == 2) return go(block_norm_grad_kernel<TX, TY, V, 2>, smem);
      return go(block_norm_grad_kernel<TX, TY, V, 4>, smem);
    });
    if (e != cudaSuccess) return e;
  }
  if (!want) return cudaSuccess;
  const int parts = a.T > 0 ? s.grid * s.rp : 0;
  return launch_pdl(norm_cols_kernel, dim3((a.H + 31) / 32), dim3(256), 0, st, a.ws, parts, a.H,
                    chan ? static_cast<const float*>(a.gate.p) : nullptr, a.gamma_post, a.post_norm, dgate_c,
                    a.dgamma_post, a.dgamma_pre);
}

}  // namespace blk
}  // namespace moe
