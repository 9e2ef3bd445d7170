// Token rows to expert order and back, with the route weights and their
// gradient.
//
// Two row movements and a dot product make up all four calls:
//   spread  out[slot(t,j)] = w_tj * tok[t]            (dispatch; collect's gradient)
//   join    out[t] = add[t] + sum_j w_tj rows[slot(t,j)]   (collect; dispatch's gradient)
//   dw_tj = <tok[t], rows[slot(t,j)]>                 (either gradient, in the same pass)
// AFN-019 "Hide SSD misses before the router knows they exist", section
// "Hypothesis H4": rows may be produced in any order into their slots, the
// weighted sum follows route-rank order.
//
// Bound by HBM: a row of every kept route moves once (spread: written, with dw
// also read; join: read) and a row of every token once.  One CTA owns a token
// (spread: up to all of its routes) and its warps share the row's pieces of
// 256 columns, so the token's row is read once whatever k is, a thread has the
// loads of eight routes in flight, and dw needs no atomics: each warp reduces
// its columns' products and the CTA adds the warps in order.
#include <algorithm>

#include "launch.h"
#include "rows.cuh"

namespace moe {
namespace blk {

namespace {

constexpr int kBatch = 8;      // routes whose loads a thread has in flight
constexpr int kMaxWarps = 16;  // warps per CTA

// Sums of eight values over the warp, each lane giving its eight: lane l
// returns the sum of value l / 4.  Three halving exchanges (4 + 2 + 1
// shuffles) leave one value per lane, two more add the four lanes of a value.
__device__ __forceinline__ float warp_sum8(const float (&v)[8], int lane) {
  float a[4], b[2];
  const bool h16 = lane & 16, h8 = lane & 8, h4 = lane & 4;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    a[i] = (h16 ? v[i + 4] : v[i]) + __shfl_xor_sync(0xffffffffu, h16 ? v[i] : v[i + 4], 16);
#pragma unroll
  for (int i = 0; i < 2; ++i) b[i] = (h8 ? a[i + 2] : a[i]) + __shfl_xor_sync(0xffffffffu, h8 ? a[i] : a[i + 2], 8);
  float c = (h4 ? b[1] : b[0]) + __shfl_xor_sync(0xffffffffu, h4 ? b[0] : b[1], 4);
  c += __shfl_xor_sync(0xffffffffu, c, 2);
  c += __shfl_xor_sync(0xffffffffu, c, 1);
  return c;
}

// A CTA's routes: slots (-1 where there is none) and weights.
struct Routes {
  int slot[kMaxK];
  float w[kMaxK];
};

__device__ __forceinline__ void read_routes(Routes& sh, const int32_t* slot_of, const float* w, size_t r0, int n,
                                            int R, int32_t* status) {
  if (threadIdx.x < n) {
    int s = slot_of[r0 + threadIdx.x];
    if (s < 0 || s >= R) {
      if (s != -1) set_status(status, MOE_DEV_BAD_EXPERT);
      s = -1;
    }
    sh.slot[threadIdx.x] = s;
    sh.w[threadIdx.x] = w != nullptr ? w[r0 + threadIdx.x] : 1.0f;
  }
  __syncthreads();
}

// dw of a CTA's n routes: the warps' sums, added in warp order.
template <int NB>
__device__ __forceinline__ void write_dw(const float (&part)[NB][kBatch], float (*red)[kMaxK], const Routes& sh,
                                         float* dw, int n) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const float s = warp_sum8(part[b], lane);
    if ((lane & 3) == 0) red[warp][b * kBatch + (lane >> 2)] = s;
  }
  __syncthreads();
  if (threadIdx.x < n) {
    float s = 0.f;
    for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i) s += red[i][threadIdx.x];
    dw[threadIdx.x] = sh.slot[threadIdx.x] < 0 ? 0.f : s;
  }
}

// NB: batches of eight routes per CTA.  grid (token, group of jb routes).
template <typename TT, typename TR, bool VEC, bool DOT, int NB>
__global__ void __launch_bounds__(kMaxWarps * 32)
    spread_kernel(const TT* tok, int64_t ld_tok, const TR* dot, int64_t ld_dot, const int32_t* __restrict__ slot_of,
                  const float* __restrict__ w, int k, int jb, int H, int R, TR* out, int64_t ld_out, float* dw,
                  int32_t* status) {
  __shared__ Routes sh;
  __shared__ float red[DOT ? kMaxWarps : 1][kMaxK];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int j0 = blockIdx.y * jb;
  const int n = min(jb, k - j0);
  const size_t r0 = static_cast<size_t>(blockIdx.x) * k + j0;
  read_routes(sh, slot_of, w, r0, n, R, status);
  const TT* row = tok + static_cast<int64_t>(blockIdx.x) * ld_tok;
  float part[DOT ? NB : 1][kBatch];
#pragma unroll
  for (int b = 0; b < (DOT ? NB : 1); ++b)
#pragma unroll
    for (int u = 0; u < kBatch; ++u) part[b][u] = 0.f;
  for (int base = warp * 256; base < H; base += warps * 256) {
    const Cols<VEC> c(base, lane, 32);
    Raw8<TT> xr;
    load8<VEC>(row, c, H, xr);
    float x[8];
    unpack(xr, x);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if (b * kBatch >= n) break;
      Raw8<TR> v[DOT ? kBatch : 1];
      if (DOT) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int j = b * kBatch + u;
          const int s = j < n ? sh.slot[j] : -1;
          if (s >= 0)
            load8<VEC>(dot + s * ld_dot, c, H, v[DOT ? u : 0]);
          else
            raw_zero(v[DOT ? u : 0]);
        }
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int j = b * kBatch + u;
        const int s = j < n ? sh.slot[j] : -1;
        if (s < 0) continue;
        if (DOT) {
          float y[8];
          unpack(v[DOT ? u : 0], y);
#pragma unroll
          for (int i = 0; i < 8; ++i) part[DOT ? b : 0][u] = fmaf(x[i], y[i], part[DOT ? b : 0][u]);
        }
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = sh.w[j] * x[i];
        store8<VEC>(out + s * ld_out, c, H, o);
      }
    }
  }
  if (DOT) write_dw<DOT ? NB : 1>(part, red, sh, dw + r0, n);
}

// grid (token, part of the columns); with DOT a token's columns stay in one CTA.
template <typename TR, typename TO, bool VEC, bool DOT, int NB>
__global__ void __launch_bounds__(kMaxWarps * 32)
    join_kernel(const TR* rows, int64_t ld_rows, const TR* dot, int64_t ld_dot, const int32_t* __restrict__ slot_of,
                const float* __restrict__ w, int k, int H, int R, TO* out, int64_t ld_out, const TO* add,
                int64_t ld_add, float* dw, int32_t* status) {
  __shared__ Routes sh;
  __shared__ float red[DOT ? kMaxWarps : 1][kMaxK];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int64_t t = blockIdx.x;
  read_routes(sh, slot_of, w, static_cast<size_t>(t) * k, k, R, blockIdx.y == 0 ? status : nullptr);
  float part[DOT ? NB : 1][kBatch];
#pragma unroll
  for (int b = 0; b < (DOT ? NB : 1); ++b)
#pragma unroll
    for (int u = 0; u < kBatch; ++u) part[b][u] = 0.f;
  for (int base = (blockIdx.y * warps + warp) * 256; base < H; base += gridDim.y * warps * 256) {
    const Cols<VEC> c(base, lane, 32);
    float x[8], acc[8];
    if (DOT) {
      Raw8<TR> xr;
      load8<VEC>(dot + t * ld_dot, c, H, xr);
      unpack(xr, x);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if (b * kBatch >= k) break;
      Raw8<TR> v[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int j = b * kBatch + u;
        const int s = j < k ? sh.slot[j] : -1;
        if (s >= 0)
          load8<VEC>(rows + s * ld_rows, c, H, v[u]);
        else
          raw_zero(v[u]);
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int j = b * kBatch + u;
        if (j >= k || sh.slot[j] < 0) continue;
        float y[8];
        unpack(v[u], y);
        const float wj = sh.w[j];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          acc[i] = fmaf(wj, y[i], acc[i]);
          if (DOT) part[DOT ? b : 0][u] = fmaf(x[i], y[i], part[DOT ? b : 0][u]);
        }
      }
    }
    if (add != nullptr) {
      Raw8<TO> ar;
      load8<VEC>(add + t * ld_add, c, H, ar);
      float a[8];
      unpack(ar, a);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += a[i];
    }
    store8<VEC>(out + t * ld_out, c, H, acc);
  }
  if (DOT) write_dw<DOT ? NB : 1>(part, red, sh, dw + static_cast<size_t>(t) * k, k);
}

int warps_for(int H) { return std::min(kMaxWarps, (H + 255) / 256); }

template <typename TT, typename TR, bool VEC, bool DOT>
cudaError_t spread(const Rows& tok, const Rows& dot, const int32_t* slot_of, const float* w, int T, int k, int H,
                   int R, const Rows& out, float* dw, int32_t* status, cudaStream_t st) {
  const int warps = warps_for(H);
  // few tokens: a token's routes are spread over several CTAs
  const int want = 4 * sm_count();
  const int jb = T >= want ? k : std::max<int64_t>(1, static_cast<int64_t>(k) * T / want);
  const dim3 grid(T, (k + jb - 1) / jb);
  auto go = [&](auto kern) {
    return launch_pdl(kern, grid, dim3(warps * 32), 0, st, static_cast<const TT*>(tok.p), tok.ld,
                      static_cast<const TR*>(dot.p), dot.ld, slot_of, w, k, jb, H, R, static_cast<TR*>(out.p), out.ld,
                      dw, status);
  };
  if (jb <= 16) return go(spread_kernel<TT, TR, VEC, DOT, 2>);
  return go(spread_kernel<TT, TR, VEC, DOT, 4>);
}

template <typename TR, typename TO, bool VEC, bool DOT>
cudaError_t join(const Rows& rows, const Rows& dot, const int32_t* slot_of, const float* w, int T, int k, int H, int R,
                 const Rows& out, const Rows& add, float* dw, int32_t* status, cudaStream_t st) {
  const int pieces = (H + 255) / 256;
  int warps = warps_for(H);
  int parts = 1;
  if (!DOT && T < 4 * sm_count()) {  // few tokens: a token's columns are spread over several CTAs
    warps = 1;
    parts = std::min(pieces, 1024);
  }
  const dim3 grid(T, parts);
  auto go = [&](auto kern) {
    return launch_pdl(kern, grid, dim3(warps * 32), 0, st, static_cast<const TR*>(rows.p), rows.ld,
                      static_cast<const TR*>(dot.p), dot.ld, slot_of, w, k, H, R, static_cast<TO*>(out.p), out.ld,
                      static_cast<const TO*>(add.p), add.ld, dw, status);
  };
  if (k <= 16) return go(join_kernel<TR, TO, VEC, DOT, 2>);
  return go(join_kernel<TR, TO, VEC, DOT, 4>);
}

// f(type tag of a, type tag of b)
template <typename F>
cudaError_t by_types(int a, int b, F&& f) {
  if (a == MOE_ROW_F32) return b == MOE_ROW_F32 ? f(float(), float()) : f(float(), bf16_t());
  return b == MOE_ROW_F32 ? f(bf16_t(), float()) : f(bf16_t(), bf16_t());
}

}  // namespace

cudaError_t launch_spread(const Rows& tok, const Rows& dot, const int32_t* slot_of, const float* w, int T, int k,
                          int H, int R, const Rows& out, float* dw, int32_t* status, cudaStream_t st) {
  const bool vec = vec_ok(tok) && vec_ok(out) && (dw == nullptr || vec_ok(dot));
  return by_types(tok.type, out.type, [&](auto tt, auto tr) {
    using TT = decltype(tt);
    using TR = decltype(tr);
    if (dw != nullptr)
      return vec ? spread<TT, TR, true, true>(tok, dot, slot_of, w, T, k, H, R, out, dw, status, st)
                 : spread<TT, TR, false, true>(tok, dot, slot_of, w, T, k, H, R, out, dw, status, st);
    return vec ? spread<TT, TR, true, false>(tok, dot, slot_of, w, T, k, H, R, out, dw, status, st)
               : spread<TT, TR, false, false>(tok, dot, slot_of, w, T, k, H, R, out, dw, status, st);
  });
}

cudaError_t launch_join(const Rows& rows, const Rows& dot, const int32_t* slot_of, const float* w, int T, int k,
                        int H, int R, const Rows& out, const Rows& add, float* dw, int32_t* status, cudaStream_t st) {
  const bool vec = vec_ok(rows) && vec_ok(out) && vec_ok(add) && (dw == nullptr || vec_ok(dot));
  return by_types(rows.type, out.type, [&](auto tr, auto to) {
    using TR = decltype(tr);
    using TO = decltype(to);
    if (dw != nullptr)
      return vec ? join<TR, TO, true, true>(rows, dot, slot_of, w, T, k, H, R, out, add, dw, status, st)
                 : join<TR, TO, false, true>(rows, dot, slot_of, w, T, k, H, R, out, add, dw, status, st);
    return vec ? join<TR, TO, true, false>(rows, dot, slot_of, w, T, k, H, R, out, add, dw, status, st)
               : join<TR, TO, false, false>(rows, dot, slot_of, w, T, k, H, R, out, add, dw, status, st);
  });
}

}  // namespace blk
}  // namespace moe
