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
// row; the row ahead is staged in shared memory (stage.cuh), with c1 and c2
// beside the stages.  fp32 stream, bf16 block, width 2,560: 24 us at 4,096 rows
// (77 % of the measured copy rate), 81 us at 16,384 (91 %): 4.6 ns a row (98 %)
// and 5 us of start and end.  Rows of 1,024 x 9,000 (unstaged) take 77 us, of
// 1,024 x 8,192 23.
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
  constexpr bool STAGED = NCH <= kMaxStagedChunks, BY_CHUNKS = kByChunks<G>;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ __align__(16) float red[15][2][16];
  const int nt = p.nt, H = a.H;
  const int group = threadIdx.x / nt, tid = threadIdx.x - group * nt;
  const bool has_y = a.y.p != nullptr, has_n = a.n_out.p != nullptr;
  // zeros where nothing is copied: without a block before it y is a row of
  // zeros, and chunks end with the row
  stage_init(red, smem, BY_CHUNKS || !has_y ? p.smem : 0);
  pdl_wait();
  pdl_trigger();
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
  const int off_y = region<TX, G, NCH>(nt), off_g = off_y + region<TY, G, NCH>(nt);
  const int64_t step = static_cast<int64_t>(gridDim.x) * p.groups;
  int64_t t = static_cast<int64_t>(blockIdx.x) * p.groups + group;
  // the thread's first place of each operand, in the group's first stage
  unsigned char* mine = smem + static_cast<size_t>(group) * p.stages * p.stage;
  unsigned char *mx = mine + tid * (G * sizeof(TX)), *my = mine + tid * (G * sizeof(TY));
  auto s_x = first_column<const TX>(a.x, t, tid * G);
  auto s_y = first_column<const TY>(a.y, t, tid * G), s_g = first_column<const TY>(a.gate, t, tid * G);
  auto w_x = first_column<TX>(a.x_out, t, tid * G);
  auto w_n = first_column<TY>(a.n_out, t, tid * G);
  int64_t ahead = t;  // the row that is staged next
  auto stage = [&](int at) {
    if (ahead < a.T) {
      stage_row<TX, G, NCH>(mx + at, s_x, tid, nt, H);
      if (has_y) stage_row<TY, G, NCH>(my + at + off_y, s_y, tid, nt, H);
      if (full) stage_row<TY, G, NCH>(my + at + off_g, s_g, tid, nt, H);
    }
    ahead += step;
    advance(s_x, p.by[0]);
    advance(s_y, p.by[1]);
    if (full) advance(s_g, p.by[2]);
    copies_commit();
  };
  if (STAGED && p.stages == 2) stage(0);
  float gt_next = token && t < a.T ? gate_v[t] : 1.0f;
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
  for (; t < a.T; t += step, advance(w_x, p.by[3]), advance(w_n, p.by[4])) {
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
    const float gt = gt_next;
    if (token && t + step < a.T) gt_next = gate_v[t + step];
    auto read_y = [&](int h, V8& f) {
      if (STAGED)
        read_staged<TY, G>(ay + off_y, y + t * a.y.ld, h, nt, f);
      else
        read_global<TY, G>(has_y ? y + t * a.y.ld : y, h, tid, nt, has_y ? H : 0, f);
    };
    V8 f;  // y, held between its two uses where a thread has eight columns
    if (NCH == 1) read_y(0, f);
    float r1 = 1.0f;
    if (a.post_norm) {
      float2 ss = splat(0.f);
#pragma unroll
      for (int h = 0; h < NCH; ++h) {
        if (NCH > 1) read_y(h, f);
        dot8(f, f, ss);
      }
      r1 = 1.0f / sqrtf(group_sum(ss.x + ss.y, red[group], which, tid, nt, group) * inv_h + a.eps);
      if (tid == 0 && a.rstd_post != nullptr) a.rstd_post[t] = r1;
    }
    V8 xo[NCH];
    float2 ss = splat(0.f);
#pragma unroll
    for (int h = 0; h < NCH; ++h) {
      if (STAGED)
        read_staged<TX, G>(ax, x + t * a.x.ld, h, nt, xo[h]);
      else
        read_global<TX, G>(x + t * a.x.ld, h, tid, nt, H, xo[h]);
      if (NCH > 1) read_y(h, f);
      V8 c;
      read_c(m1, h, c);
      // y r1 first: the normalised value, which no gate can overflow
      f = f * r1 * gt;
      if (full) {
        V8 g;
        if (STAGED)
          read_staged<TY, G>(ay + off_g, gate + t * a.gate.ld, h, nt, g);
        else
          read_global<TY, G>(gate + t * a.gate.ld, h, tid, nt, H, g);
        f = f * g;
      }
      xo[h] = fma8(f, c, xo[h] * a.scale);
      dot8(xo[h], xo[h], ss);
      if (a.x_out.p != nullptr) write_row<TX, G>(w_x, h, tid, nt, H, xo[h]);
    }
    if (!has_n) continue;
    const float r2 = 1.0f / sqrtf(group_sum(ss.x + ss.y, red[group], which, tid, nt, group) * inv_h + a.eps);
    if (tid == 0 && a.rstd_pre != nullptr) a.rstd_pre[t] = r2;
#pragma unroll
    for (int h = 0; h < NCH; ++h) {
      V8 c;
      read_c(m2, h, c);
      xo[h] = xo[h] * r2 * c;
      write_row<TY, G>(w_n, h, tid, nt, H, xo[h]);
    }
  }
}

}  // namespace

cudaError_t launch_block_norm(const NormArgs& a, cudaStream_t st) {
  const bool full = a.gate_kind == MOE_GATE_FULL;
  const Rows gate = full ? a.gate : Rows{nullptr, 0, MOE_ROW_F32};
  const int unit = norm_unit(a.H, {a.x, a.y, gate, a.x_out, a.n_out});
  NormPlan p = norm_plan(a.T, a.H, row_bytes8(a.x) + (a.y.type == MOE_ROW_F32 ? 32 : 16) + row_bytes8(gate),
                         unit == 1 ? 3 : 0, kThreads);
  plan_steps(p, {a.x, a.y, gate, a.x_out, a.n_out});
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
