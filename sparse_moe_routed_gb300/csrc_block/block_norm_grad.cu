// Gradient of the block norm (block_norm.cu).
//
// With xh = x_out r2, yh = y r1 (the normalised rows), u = dn c2, c1 = (1 +
// gamma_post) times a per-channel gate and g the gate where it varies by row:
//   D  = dx_out + r2 (u - xh mean(u xh)),   dx = scale D
//   q  = sum D c1 yh,   dy = r1 g (D c1 - yh q / H),   per-token dgate = q
// (a gate per element goes into D before q instead).
// Written with normalised rows, so that a small row's large r is never cubed.
// Per column, A = sum_t D g yh gives dgamma_post = gate_c A as well as a
// per-channel dgate = (1 + gamma_post) A, and B = sum_t dn xh is dgamma_pre:
// two accumulators per column, whatever the gate.
//
// Bound by HBM: four rows in, two out.  A group of threads owns a row, the row
// ahead is staged in shared memory (stage.cuh); where a thread has eight
// columns it holds the normalised rows between the row's three steps, else it
// reads the stage again.  One CTA per SM keeps A and B over all its rows and
// writes one partial row of each; a second launch adds these in order.  fp32
// stream, bf16 block, width 2,560: 39 us at 4,096 rows (72 % of the measured
// copy rate), 118 us at 16,384 (94 %): 6.5 ns a row and 10 us that do not grow
// with the rows, 6 of them the column sums with their launch (at 1,024, 4,096
// and 16,384 rows alike), the rest start and first rows.  Rows of 1,024 x 9,000
// (unstaged) take 214 us, of 1,024 x 8,192 50.
#include <math.h>

#include "norm.h"
#include "stage.cuh"

namespace moe {
namespace blk {

namespace {

// 96 registers a thread: spills would miss the small L1 that the stages leave
// (a form that spilled six registers per row took 56 us, not 46).  The forms of
// eight columns per thread spill up to 36 bytes, those of wider rows 224 to 752.
constexpr int kThreads = 640;

template <typename TX, typename TY, int G, int NCH>
__global__ void __launch_bounds__(NCH == 1 ? kThreads : kMaxGroupThreads)
    block_norm_grad_kernel(const NormGradArgs a, const NormPlan p, int want_cols) {
  constexpr bool STAGED = NCH <= kMaxStagedChunks, BY_CHUNKS = kByChunks<G>;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ __align__(16) float red[15][2][16];
  const int nt = p.nt, H = a.H;
  const int group = threadIdx.x / nt, tid = threadIdx.x - group * nt;
  const bool has_d = a.dx_out.p != nullptr, has_n = a.dn.p != nullptr, has_y = a.y.p != nullptr;
  // zeros where nothing is copied: an absent gradient is a row of zeros, and
  // chunks end with the row
  stage_init(red, smem, BY_CHUNKS || !has_d || !has_n ? p.smem : 0);
  pdl_wait();
  pdl_trigger();
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
  // c1 and c2 of every column behind the stages, laid out like fp32 rows;
  // unstaged kernels read them from global memory
  unsigned char* m1 = smem + static_cast<size_t>(p.groups) * p.stages * p.stage + tid * (G * 4);
  unsigned char* m2 = m1 + NCH * nt * 32;
  auto read_c = [&](const unsigned char* m, int h, V8& f) {
    if (STAGED) {
      read_staged<float, G>(m, nullptr, h, nt, f);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = col0<G>(h, i, tid, nt);
        el(f, i) = c >= H ? 0.f : m == m1 ? c1_at(c) : gain(a.gamma_pre, c);
      }
    }
  };
  // column sums: registers, or (unstaged, widest rows) the thread's own
  // places in shared memory
  constexpr int NA = STAGED ? NCH : 1;
  V8 accA[NA], accB[NA];
#pragma unroll
  for (int h = 0; h < NA; ++h)
#pragma unroll
    for (int i = 0; i < 4; ++i) accA[h].v[i] = accB[h].v[i] = splat(0.f);
  float* shA = reinterpret_cast<float*>(smem) + tid;
  float* shB = shA + NCH * 8 * nt;
  if (!STAGED)
    for (int i = 0; i < NCH * 8; ++i) shA[i * nt] = shB[i * nt] = 0.f;
  // acc += v w for chunk h
  auto add_cols = [&](V8(&acc)[NA], float* sh, int h, const V8& v, float w) {
    if (STAGED) {
      acc[STAGED ? h : 0] = fma8(v, w, acc[STAGED ? h : 0]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) sh[(h * 8 + i) * nt] = fmaf(el(v, i), w, sh[(h * 8 + i) * nt]);
    }
  };

  const int bx = region<TX, G, NCH>(nt), by = region<TY, G, NCH>(nt);
  const int off_x = bx, off_dn = off_x + bx, off_y = off_dn + by, off_g = off_y + (has_y ? by : 0);
  const int64_t step = static_cast<int64_t>(gridDim.x) * p.groups;
  int64_t t = static_cast<int64_t>(blockIdx.x) * p.groups + group;
  // the thread's first place of each operand, in the group's first stage
  unsigned char* mine = smem + static_cast<size_t>(group) * p.stages * p.stage;
  unsigned char *mx = mine + tid * (G * sizeof(TX)), *my = mine + tid * (G * sizeof(TY));
  auto s_dxo = first_column<const TX>(a.dx_out, t, tid * G), s_xo = first_column<const TX>(a.x_out, t, tid * G);
  auto s_dn = first_column<const TY>(a.dn, t, tid * G), s_y = first_column<const TY>(a.y, t, tid * G),
       s_g = first_column<const TY>(a.gate, t, tid * G);
  auto w_dx = first_column<TX>(a.dx, t, tid * G);
  auto w_dy = first_column<TY>(a.dy, t, tid * G);
  int64_t ahead = t;  // the row that is staged next
  auto stage = [&](int at) {
    if (ahead < a.T) {
      if (has_d) stage_row<TX, G, NCH>(mx + at, s_dxo, tid, nt, H);
      if (has_n) {
        stage_row<TX, G, NCH>(mx + at + off_x, s_xo, tid, nt, H);
        stage_row<TY, G, NCH>(my + at + off_dn, s_dn, tid, nt, H);
      }
      if (has_y) stage_row<TY, G, NCH>(my + at + off_y, s_y, tid, nt, H);
      if (full) stage_row<TY, G, NCH>(my + at + off_g, s_g, tid, nt, H);
    }
    ahead += step;
    advance(s_dxo, p.by[0]);
    advance(s_xo, p.by[1]);
    advance(s_dn, p.by[2]);
    advance(s_y, p.by[3]);
    if (full) advance(s_g, p.by[4]);
    copies_commit();
  };
  if (STAGED && p.stages == 2) stage(0);
  float r1n = 1.f, r2n = 0.f, gtn = 1.f;  // the next row's factors
  auto factors = [&](int64_t row) {
    if (row >= a.T) return;
    if (a.post_norm) r1n = a.rstd_post[row];
    if (has_n) r2n = a.rstd_pre[row];
    if (token) gtn = gate_v[row];
  };
  factors(t);
  // after the first rows' copies are on their way
  if (STAGED) {
    // place i holds column i: units of G columns are adjacent
    float* g = reinterpret_cast<float*>(smem + static_cast<size_t>(p.groups) * p.stages * p.stage);
    for (int i0 = threadIdx.x; i0 < NCH * 8 * nt; i0 += 8 * blockDim.x) {
      float v1[8], v2[8];  // eight columns' loads in flight
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i = i0 + k * blockDim.x;
        v1[k] = i < H ? c1_at(i) : 0.f;
        v2[k] = i < H ? gain(a.gamma_pre, i) : 0.f;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i = i0 + k * blockDim.x;
        if (i < NCH * 8 * nt) g[i] = v1[k], g[NCH * 8 * nt + i] = v2[k];
      }
    }
    __syncthreads();
  }
  int which = 0, at = 0;
  for (; t < a.T; t += step, advance(w_dx, p.by[5]), advance(w_dy, p.by[6])) {
    const unsigned char *ax = mx + at, *ay = my + at;
    if (STAGED) {
      if (p.stages == 1) {
        if (BY_CHUNKS) group_sync(nt, group);  // the row before has been read
        stage(0);
      }
      copies_wait();
      if (BY_CHUNKS) group_sync(nt, group);  // this row is there, and with two stages the one before has been read
      if (p.stages == 2) stage(p.stage - at);
      at = p.stages == 2 ? p.stage - at : 0;
    }
    const float r1 = r1n, r2 = r2n, gt = gtn;
    factors(t + step);
    auto read_x = [&](int off, const TX* q, int64_t ld, int h, V8& f) {
      if (STAGED)
        read_staged<TX, G>(ax + off, q + t * ld, h, nt, f);
      else
        read_global<TX, G>(q == nullptr ? q : q + t * ld, h, tid, nt, q == nullptr ? 0 : H, f);
    };
    auto read_y = [&](int off, const TY* q, int64_t ld, int h, V8& f) {
      if (STAGED)
        read_staged<TY, G>(ay + off, q + t * ld, h, nt, f);
      else
        read_global<TY, G>(q == nullptr ? q : q + t * ld, h, tid, nt, q == nullptr ? 0 : H, f);
    };
    // where a thread has eight columns, xh, u = dn c2 and yh are held between
    // the row's steps; wider rows are read again
    V8 xh, u, yh;
    float2 dot = splat(0.f);
#pragma unroll
    for (int h = 0; h < NCH; ++h) {
      V8 c;
      read_c(m2, h, c);
      read_x(off_x, xo, a.x_out.ld, h, xh);
      read_y(off_dn, dn, a.dn.ld, h, u);
      xh = xh * r2;
      add_cols(accB, shB, h, u * xh, 1.0f);
      u = u * c;
      dot8(u, xh, dot);
    }
    float m = group_sum(dot.x + dot.y, red[group], which, tid, nt, group) * inv_h;

    V8 D[NCH];
    float2 qs = splat(0.f);
#pragma unroll
    for (int h = 0; h < NCH; ++h) {
      V8 c;
      if (NCH > 1) {
        read_c(m2, h, c);
        read_x(off_x, xo, a.x_out.ld, h, xh);
        read_y(off_dn, dn, a.dn.ld, h, u);
        xh = xh * r2;
        u = u * c;
      }
      read_x(0, dxo, a.dx_out.ld, h, D[h]);
      D[h] = fma8(fma8(xh, -m, u), r2, D[h]);
      write_row<TX, G>(w_dx, h, tid, nt, H, D[h] * a.scale);
      if (!has_y) continue;
      read_y(off_y, y, a.y.ld, h, yh);
      yh = yh * r1;
      read_c(m1, h, c);
      if (full) {
        V8 g;
        read_y(off_g, gate, a.gate.ld, h, g);
        if (a.dgate.p != nullptr)
          write_row<TY, G>(static_cast<TY*>(a.dgate.p) + t * a.dgate.ld + tid * G, h, tid, nt, H, D[h] * c * yh);
        D[h] = D[h] * g;
      }
      const V8 v = D[h] * yh;
      add_cols(accA, shA, h, v, gt);
      dot8(v, c, qs);
      D[h] = D[h] * c;
    }
    if (!has_y) continue;
    float q = qs.x + qs.y;
    if (a.post_norm || token) {
      q = group_sum(q, red[group], which, tid, nt, group);
      if (token && tid == 0 && a.dgate.p != nullptr) static_cast<float*>(a.dgate.p)[t] = q;
    }
    m = q * inv_h;
    const float rg = r1 * gt;
#pragma unroll
    for (int h = 0; h < NCH; ++h) {
      if (a.post_norm) {
        if (NCH > 1) {
          read_y(off_y, y, a.y.ld, h, yh);
          yh = yh * r1;
        }
        D[h] = fma8(yh, -m, D[h]);
      }
      write_row<TY, G>(w_dy, h, tid, nt, H, D[h] * rg);
    }
  }
  if (!want_cols) return;
  // the groups' sums, added in group order, then one partial row of A and B
  if (STAGED && p.groups > 1) {
    float* sh = reinterpret_cast<float*>(smem);
    __syncthreads();
    if (group > 0) {
      float* s = sh + static_cast<size_t>(group - 1) * 16 * NA * nt + tid;
#pragma unroll
      for (int i = 0; i < 8 * NA; ++i) {
        s[i * nt] = el(accA[i / 8], i % 8);
        s[(8 * NA + i) * nt] = el(accB[i / 8], i % 8);
      }
    }
    __syncthreads();
    if (group > 0) return;
    for (int k = 0; k + 1 < p.groups; ++k) {
      const float* s = sh + static_cast<size_t>(k) * 16 * NA * nt + tid;
#pragma unroll
      for (int i = 0; i < 8 * NA; ++i) {
        el(accA[i / 8], i % 8) += s[i * nt];
        el(accB[i / 8], i % 8) += s[(8 * NA + i) * nt];
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
      w[c] = STAGED ? el(accA[STAGED ? h : 0], i) : shA[(h * 8 + i) * nt];
      w[H + c] = STAGED ? el(accB[STAGED ? h : 0], i) : shB[(h * 8 + i) * nt];
    }
}

// Column sums over the parts: 32 columns by 32 threads, each of which adds
// every 32nd part in order, then these in order.  blockIdx.y 0: A, 1: B.
__global__ void __launch_bounds__(1024) norm_cols_kernel(const float* __restrict__ ws, int parts, int H,
                                                         const float* gate_c, const float* gamma_post, int post_norm,
                                                         float* dgate_c, float* dgamma_post, float* dgamma_pre) {
  __shared__ float sh[32][33];
  pdl_wait();
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + tx;
  const float* w = ws + blockIdx.y * H + col;
  float v = 0.f;
  if (col < H) {
#pragma unroll 8
    for (int p = ty; p < parts; p += 32) v += w[static_cast<size_t>(p) * 2 * H];
  }
  sh[ty][tx] = v;
  __syncthreads();
  // warp ty adds column ty's 32 sums
  v = sh[tx][ty];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int c = blockIdx.x * 32 + ty;
  if (tx != 0 || c >= H) return;
  if (blockIdx.y == 1) {
    if (dgamma_pre != nullptr) dgamma_pre[c] = v;
    return;
  }
  // no rows: zero, whatever the gate and the gain hold
  if (dgamma_post != nullptr) dgamma_post[c] = gate_c != nullptr && parts > 0 ? gate_c[c] * v : v;
  if (dgate_c != nullptr) dgate_c[c] = post_norm && parts > 0 ? gain(gamma_post, c) * v : v;
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
    const int sx = a.dx.type == MOE_ROW_F32 ? 32 : 16, sy = a.y.type == MOE_ROW_F32 ? 32 : 16;
    const int slot = 2 * sx + sy + row_bytes8(a.y) + row_bytes8(gate);
    const int unit = norm_unit(a.H, {a.dx_out, a.x_out, a.dn, a.y, gate, dgate, a.dx, a.dy});
    NormPlan p = norm_plan(a.T, a.H, slot, unit == 1 ? 5 : 0, kThreads);
    p.grid = std::min(p.grid, sm_count());
    const int cols = p.nch <= kMaxStagedChunks ? (p.groups - 1) * 2 * p.nch * 8 * p.nt * 4 : 2 * p.nch * 8 * p.nt * 4;
    p.smem = std::max(p.smem, cols);  // the sums' join takes the stages' place
    parts = p.grid;
    plan_steps(p, {a.dx_out, a.x_out, a.dn, a.y, gate, a.dx, a.dy});
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
  return launch_pdl(norm_cols_kernel, dim3((a.H + 31) / 32, 2), dim3(1024), 0, st, a.ws, parts, a.H,
                    chan ? static_cast<const float*>(a.gate.p) : nullptr, a.gamma_post, a.post_norm, dgate_c,
                    a.dgamma_post, a.dgamma_pre);
}

}  // namespace blk
}  // namespace moe
