// The experts' feed-forward block for training, and its gradient: six
// contractions per expert, from operands in shared memory on the CUDA cores.
#include <algorithm>

#include "launch.h"
#include "q8.cuh"
#include "rows.cuh"

namespace moe {
namespace blk {

namespace {

constexpr int kTile = 64, kStep = 16;

struct P {
  const uint16_t *a, *b;  // operands: a weights (weight gradients: the output's rows)
  int64_t lda, ldb;
  const int32_t* offsets;
  int R, E, H, I;
  void* out;
  int64_t ld_out;
  int out_type, accumulate;
  Act act;
  uint16_t *da, *h;
};

enum { kGateUp, kDown, kDh, kDx, kDwGateUp, kDwDown };

__device__ __forceinline__ int seg(const P& p, int e) { return min(max(p.offsets[e], 0), p.R); }

__device__ __forceinline__ void put_any(void* out, int type, int64_t i, float v, int accumulate) {
  if (type == MOE_ROW_F32) {
    float* o = static_cast<float*>(out) + i;
    *o = accumulate ? *o + v : v;
  } else {
    uint16_t* o = static_cast<uint16_t*>(out) + i;
    *o = f32_to_bf16(accumulate ? bf16_to_f32(*o) + v : v);
  }
}

// grid (tiles of m, [tiles of n,] experts).  m: features; n: the expert's slots, or for a weight gradient the
// output's columns, with the slots as k.
template <int MODE>
__global__ void __launch_bounds__(256) ffn_simple_kernel(P p) {
  __shared__ float sa[kStep][kTile + 1], sb[kStep][kTile + 1], sc[kTile][kTile + 1];
  pdl_wait();
  constexpr bool kW = MODE == kDwGateUp || MODE == kDwDown;
  const int e = kW ? blockIdx.z : blockIdx.y, tid = threadIdx.x;
  const int s0 = seg(p, e), n_e = max(seg(p, e + 1) - s0, 0);
  const int I = p.I, H = p.H;
  const int M = MODE == kGateUp || MODE == kDwGateUp ? 2 * I : MODE == kDh ? I : H;
  const int K = kW ? n_e : MODE == kGateUp || MODE == kDh ? H : MODE == kDown ? I : 2 * I;
  const int N = kW ? (MODE == kDwGateUp ? H : I) : n_e;
  const int nstep = kW ? (N + kTile - 1) / kTile * kTile : kTile;
  for (int n0 = kW ? blockIdx.y * kTile : 0; n0 < N; n0 += nstep) {
    float acc[4][4] = {};
    for (int k0 = 0; k0 < K; k0 += kStep) {
      for (int i = tid; i < kTile * kStep; i += 256) {
        const int r = MODE == kGateUp || MODE == kDown ? i / kStep : i % kTile;
        const int c = MODE == kGateUp || MODE == kDown ? i % kStep : i / kTile;
        const int k = k0 + c;
        int m = blockIdx.x * kTile + r;
        if (MODE == kGateUp) m = r < 32 ? blockIdx.x * 32 + r : I + blockIdx.x * 32 + r - 32;  // a gate half and its up half
        const bool in = k < K && (MODE == kGateUp ? blockIdx.x * 32 + (r & 31) < I : m < M);
        int64_t at;
        if (MODE == kGateUp || MODE == kDown)
          at = (static_cast<int64_t>(e) * M + m) * K + k;
        else if (!kW)
          at = (static_cast<int64_t>(e) * K + k) * M + m;
        else
          at = (s0 + k) * p.lda + m;
        sa[c][r] = in ? bf16_to_f32(p.a[at]) : 0.f;
        const int rb = kW ? i % kTile : i / kStep, cb = kW ? i / kTile : i % kStep;
        const int n = n0 + rb, kb = k0 + cb;
        sb[cb][rb] = n < N && kb < K ? bf16_to_f32(p.b[kW ? (s0 + kb) * p.ldb + n : (s0 + n) * p.ldb + kb]) : 0.f;
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kStep; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] += sa[k][tid % 16 + 16 * i] * sb[k][tid / 16 + 16 * j];
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) sc[tid / 16 + 16 * j][tid % 16 + 16 * i] = acc[i][j];
    __syncthreads();
    // a warp per n, its lanes along m
    for (int n = tid / 32; n < kTile && n0 + n < N; n += 8) {
      const int lane = tid & 31;
      const int64_t s = s0 + n0 + n;
      if (MODE == kGateUp) {
        const int i = blockIdx.x * 32 + lane;
        const float g = sc[n][lane], u = sc[n][lane + 32];
        if (p.act.kind == MOE_ACT_Q8) {
          const uint32_t eg = exp_byte(__reduce_max_sync(0xffffffffu, __float_as_uint(g) & 0x7fffffffu));
          const uint32_t eu = exp_byte(__reduce_max_sync(0xffffffffu, __float_as_uint(u) & 0x7fffffffu));
          const int G = (I + kGroup - 1) / kGroup;
          uint8_t* q = static_cast<uint8_t*>(p.act.p) + s * p.act.ld;
          uint8_t* ex = p.act.exp.p + s * p.act.exp.ld + blockIdx.x;
          if (i < I) q[i] = static_cast<uint8_t>(to_q8(g, inv_scale(eg))), q[I + i] = static_cast<uint8_t>(to_q8(u, inv_scale(eu)));
          if (lane == 0) ex[0] = static_cast<uint8_t>(eg), ex[G] = static_cast<uint8_t>(eu);
        }
        if (i >= I) continue;
        if (p.act.kind == MOE_ACT_BF16) {
          uint16_t* a = static_cast<uint16_t*>(p.act.p) + s * p.act.ld;
          a[i] = f32_to_bf16(g);
          a[I + i] = f32_to_bf16(u);
        }
        p.h[s * I + i] = f32_to_bf16(g / (1.f + expf(-g)) * u);
        continue;
      }
      for (int c = lane; c < kTile; c += 32) {
        const int m = blockIdx.x * kTile + c;
        if (m >= M) continue;
        const float v = sc[n][c];
        if (MODE == kDh) {
          float g, u;
          if (p.act.kind == MOE_ACT_Q8) {
            const int G = (I + kGroup - 1) / kGroup;
            const int8_t* q = static_cast<const int8_t*>(p.act.p) + s * p.act.ld;
            const uint8_t* ex = p.act.exp.p + s * p.act.exp.ld + m / kGroup;
            g = q[m] * scale_of(ex[0]);
            u = q[I + m] * scale_of(ex[G]);
          } else {
            const uint16_t* a = static_cast<const uint16_t*>(p.act.p) + s * p.act.ld;
            g = bf16_to_f32(a[m]);
            u = bf16_to_f32(a[I + m]);
          }
          const float r = 1.f / (1.f + expf(-g));
          p.da[s * 2 * I + m] = f32_to_bf16(v * u * r * (1.f + g * (1.f - r)));
          p.da[s * 2 * I + I + m] = f32_to_bf16(v * g * r);
          p.h[s * I + m] = f32_to_bf16(g * r * u);
        } else if (kW) {
          put_any(p.out, p.out_type, (static_cast<int64_t>(e) * M + m) * N + n0 + n, v, p.accumulate);
        } else {
          put_any(p.out, p.out_type, s * p.ld_out + m, v, 0);
        }
      }
    }
    __syncthreads();
  }
}

inline int up(int a, int b) { return (a + b - 1) / b; }

template <int MODE>
cudaError_t go(const P& p, cudaStream_t st) {
  const dim3 grid = MODE == kGateUp     ? dim3(up(p.I, 32), p.E)
                    : MODE == kDh       ? dim3(up(p.I, kTile), p.E)
                    : MODE == kDwGateUp ? dim3(up(2 * p.I, kTile), up(p.H, kTile), p.E)
                    : MODE == kDwDown   ? dim3(up(p.H, kTile), up(p.I, kTile), p.E)
                                        : dim3(up(p.H, kTile), p.E);
  return launch_pdl(ffn_simple_kernel<MODE>, grid, dim3(256), 0, st, p);
}

#define FFN_TRY(call)                            \
  do {                                           \
    const cudaError_t e_ = (call);               \
    if (e_ != cudaSuccess) return e_;            \
  } while (0)

}  // namespace

cudaError_t launch_ffn(const FfnArgs& a, cudaStream_t st) {
  P p{};
  p.offsets = a.offsets;
  p.R = a.R, p.E = a.E, p.H = a.H, p.I = a.I;
  p.a = a.w_gateup;
  p.b = static_cast<const uint16_t*>(a.x.p);
  p.ldb = a.x.ld;
  p.act = a.act;
  p.h = a.h;
  FFN_TRY(go<kGateUp>(p, st));
  if (a.y.p == nullptr) return cudaSuccess;
  p.a = a.w_down;
  p.b = a.h;
  p.ldb = a.I;
  p.out = a.y.p;
  p.ld_out = a.y.ld;
  p.out_type = a.y.type;
  return go<kDown>(p, st);
}

cudaError_t launch_ffn_grad(const FfnGradArgs& a, cudaStream_t st) {
  if (a.R == 0) {
    const size_t n = static_cast<size_t>(a.E) * a.H * a.I * (a.dw_type == MOE_ROW_F32 ? 4 : 2);
    if (a.dw_gateup && !a.accumulate) FFN_TRY(cudaMemsetAsync(a.dw_gateup, 0, 2 * n, st));
    if (a.dw_down && !a.accumulate) FFN_TRY(cudaMemsetAsync(a.dw_down, 0, n, st));
    return cudaSuccess;
  }
  P p{};
  p.offsets = a.offsets;
  p.R = a.R, p.E = a.E, p.H = a.H, p.I = a.I;
  p.a = a.w_down;
  p.b = static_cast<const uint16_t*>(a.dy.p);
  p.ldb = a.dy.ld;
  p.act = a.act;
  p.da = a.da;
  p.h = a.h;
  FFN_TRY(go<kDh>(p, st));
  if (a.dx.p != nullptr) {
    p.a = a.w_gateup;
    p.b = a.da;
    p.ldb = 2 * a.I;
    p.out = a.dx.p;
    p.ld_out = a.dx.ld;
    p.out_type = a.dx.type;
    FFN_TRY(go<kDx>(p, st));
  }
  p.out_type = a.dw_type;
  p.accumulate = a.accumulate;
  if (a.dw_gateup != nullptr) {
    p.a = a.da;
    p.lda = 2 * a.I;
    p.b = static_cast<const uint16_t*>(a.x.p);
    p.ldb = a.x.ld;
    p.out = a.dw_gateup;
    FFN_TRY(go<kDwGateUp>(p, st));
  }
  if (a.dw_down != nullptr) {
    p.a = static_cast<const uint16_t*>(a.dy.p);
    p.lda = a.dy.ld;
    p.b = a.h;
    p.ldb = a.I;
    p.out = a.dw_down;
    FFN_TRY(go<kDwDown>(p, st));
  }
  return cudaSuccess;
}

}  // namespace blk
}  // namespace moe
