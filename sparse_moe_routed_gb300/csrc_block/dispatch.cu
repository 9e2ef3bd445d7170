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
// also read; join: read) and a row of every token once.  With many tokens one
// warp owns a token: it walks the row's pieces of 256 columns, each lane with
// the loads of up to eight routes in flight, and needs no barrier from its
// slots to its dw.  With few, the warps of a CTA share a token's pieces (and
// CTAs its routes or columns), and dw adds the warps' sums in order.  dw needs
// no atomics in either form, and the token's row is read once whatever k is.
// Top 10, width 2,560, bf16: dispatch 36 us (90 % of the measured copy rate) and
// its gradient with dw 50 us (78 %) at 4,096 tokens, collect's gradient 270 us
// (96 %) at 16,384; of fp32 rows dispatch's gradient 84 us (96 %) at 4,096.
#include <algorithm>
#include <type_traits>

#include "launch.h"
#include "rows.cuh"

namespace moe {
namespace blk {

namespace {

// Routes whose loads a thread has in flight.  A lone warp per token wants eight
// (collect's gradient at 16,384 tokens: 269 us against 273 with four), CTAs of
// several warps are better off with four and twice the CTAs per SM (dispatch's
// gradient at 2,048 tokens: 24.7 against 33.2 us).  fp32 rows, and single
// elements, need twice the registers for a route: half of each, or what the
// launch bounds leave spills more (dispatch's gradient of fp32 rows, 4,096 tokens:
// 83.7 us with four, 128 with eight; 1,024 tokens: 25.4 with two, 29.8 with
// four, but collect without dw 20.2 with four, 21.4 with two; of odd bf16 rows,
// 4,096 tokens: 86.3 us with two, 110 with four).  Most kernels with dw still
// spill: where a warp owns a token up to 120 bytes a thread for up to 16 routes
// (48 for bf16 rows in whole pieces) and 300 above; join with several warps per
// token on odd elements 264 to 356 bytes, above 16 routes 636 to 820 (without dw
// 56 to 80).
template <bool SOLO, bool DOT, typename TR, int U>
constexpr int kBatch = sizeof(TR) == 2 && U > 1 ? (SOLO ? 8 : 4)
                       : sizeof(TR) == 4 && SOLO ? 4
                                                 : (DOT ? 2 : 4);
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

// A token's routes: where the row of each starts (-1: it has none), weights.
struct Routes {
  int64_t at[kMaxK];
  float w[kMaxK];
};

// Fills the routes with threads 0..n-1 of the token's warps.
__device__ __forceinline__ void read_routes(Routes& sh, const int32_t* slot_of, const float* w, size_t r0, int n,
                                            int tid, int R, int64_t ld, int32_t* status) {
  if (tid >= n) return;
  const int s = slot_of[r0 + tid];
  const bool ok = s >= 0 && s < R;
  if (!ok && s != -1) set_status(status, MOE_DEV_BAD_EXPERT);
  sh.at[tid] = ok ? s * ld : -1;
  sh.w[tid] = w != nullptr ? w[r0 + tid] : 1.0f;
}

// The warps of one token: SOLO, each warp of the CTA has its own token.
template <bool SOLO>
__device__ __forceinline__ void token_sync() {
  if (SOLO)
    __syncwarp();
  else
    __syncthreads();
}

// dw of a token's n routes: the warps' sums, added in warp order.
template <bool SOLO, int NB>
__device__ __forceinline__ void write_dw(const float (&part)[NB][8], float (*red)[kMaxK], const Routes& sh,
                                         float* dw, int n, int warp, int warps, int tid) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const float s = warp_sum8(part[b], lane);
    if ((lane & 3) == 0) red[warp][b * 8 + (lane >> 2)] = s;
  }
  token_sync<SOLO>();
  if (tid < n) {
    float s = red[SOLO ? warp : 0][tid];
    if (!SOLO)
      for (int i = 1; i < warps; ++i) s += red[i][tid];
    dw[tid] = sh.at[tid] < 0 ? 0.f : s;
  }
}

constexpr int kSoloWarps = 4;  // tokens per CTA where a warp owns a token

// NK: routes per CTA at most (with DOT each has a register).  SOLO: grid
// (tokens / kSoloWarps); else grid (token, group of jb routes).
template <typename TT, typename TR, int U, bool DOT, int NK, bool SOLO>
__global__ void __launch_bounds__(SOLO ? kSoloWarps * 32 : kMaxWarps * 32, SOLO ? 7 : 2)
    spread_kernel(const TT* tok, int64_t ld_tok, const TR* dot, int64_t ld_dot, const int32_t* __restrict__ slot_of,
                  const float* __restrict__ w, int T, int k, int jb, int H, int R, TR* out, int64_t ld_out, float* dw,
                  int32_t* status) {
  __shared__ Routes routes[SOLO ? kSoloWarps : 1];
  __shared__ float red[DOT ? (SOLO ? kSoloWarps : kMaxWarps) : 1][kMaxK];
  pdl_wait();
  pdl_trigger();
  constexpr int B = kBatch<SOLO, DOT, TR, U>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = SOLO ? 1 : blockDim.x >> 5;
  const int tid = SOLO ? lane : threadIdx.x;
  const int64_t t = SOLO ? static_cast<int64_t>(blockIdx.x) * kSoloWarps + warp : blockIdx.x;
  if (SOLO && t >= T) return;
  const int j0 = SOLO ? 0 : blockIdx.y * jb;
  const int n = SOLO ? k : min(jb, k - j0);
  const size_t r0 = static_cast<size_t>(t) * k + j0;
  Routes& sh = routes[SOLO ? warp : 0];
  // dot and out have rows at the same slots: their strides differ
  read_routes(sh, slot_of, w, r0, n, tid, R, 1, status);
  token_sync<SOLO>();
  const TT* row = tok + t * ld_tok;
  float part[DOT ? NK / 8 : 1][8];  // this lane's share of each route's product
#pragma unroll
  for (int b = 0; b < (DOT ? NK / 8 : 1); ++b)
#pragma unroll
    for (int u = 0; u < 8; ++u) part[b][u] = 0.f;
  for (int base = (SOLO ? 0 : warp) * 256; base < H; base += warps * 256) {
    const Cols<U> c(base, lane, 32);
    Raw8<TT> xr;
    load8<U>(row, c, H, xr);
    const V8 x = unpack(xr);
#pragma unroll
    for (int b = 0; b < NK / B; ++b) {
      if (b * B >= n) break;
      Raw8<TR> v[DOT ? B : 1];
      if (DOT) {
#pragma unroll
        for (int u = 0; u < B; ++u) {
          const int j = b * B + u;
          const int64_t s = j < n ? sh.at[j] : -1;
          if (s >= 0)
            load8<U>(dot + s * ld_dot, c, H, v[DOT ? u : 0]);
          else
            raw_zero(v[DOT ? u : 0]);
        }
      }
#pragma unroll
      for (int u = 0; u < B; ++u) {
        const int j = b * B + u;
        const int64_t s = j < n ? sh.at[j] : -1;
        if (s < 0) continue;
        if (DOT) {
          float2 p = splat(0.f);
          dot8(x, unpack(v[DOT ? u : 0]), p);
          part[DOT ? j / 8 : 0][j % 8] += p.x + p.y;
        }
        store8<U>(out + s * ld_out, c, H, x * sh.w[j]);
      }
    }
  }
  if (DOT) write_dw<SOLO, DOT ? NK / 8 : 1>(part, red, sh, dw + r0, n, warp, warps, tid);
}

// SOLO: grid (tokens / kSoloWarps); else grid (token, part of the columns),
// one part with DOT.
template <typename TR, typename TO, int U, bool DOT, int NK, bool SOLO>
__global__ void __launch_bounds__(SOLO ? kSoloWarps * 32 : kMaxWarps * 32, SOLO ? 7 : 2)
    join_kernel(const TR* rows, int64_t ld_rows, const TR* dot, int64_t ld_dot, const int32_t* __restrict__ slot_of,
                const float* __restrict__ w, int T, int k, int H, int R, TO* out, int64_t ld_out, const TO* add,
                int64_t ld_add, float* dw, int32_t* status) {
  __shared__ Routes routes[SOLO ? kSoloWarps : 1];
  __shared__ float red[DOT ? (SOLO ? kSoloWarps : kMaxWarps) : 1][kMaxK];
  pdl_wait();
  pdl_trigger();
  constexpr int B = kBatch<SOLO, DOT, TR, U>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = SOLO ? 1 : blockDim.x >> 5;
  const int tid = SOLO ? lane : threadIdx.x;
  const int64_t t = SOLO ? static_cast<int64_t>(blockIdx.x) * kSoloWarps + warp : blockIdx.x;
  if (SOLO && t >= T) return;
  Routes& sh = routes[SOLO ? warp : 0];
  const size_t r0 = static_cast<size_t>(t) * k;
  read_routes(sh, slot_of, w, r0, k, tid, R, ld_rows, SOLO || blockIdx.y == 0 ? status : nullptr);
  token_sync<SOLO>();
  float part[DOT ? NK / 8 : 1][8];  // this lane's share of each route's product
#pragma unroll
  for (int b = 0; b < (DOT ? NK / 8 : 1); ++b)
#pragma unroll
    for (int u = 0; u < 8; ++u) part[b][u] = 0.f;
  const int first = SOLO ? 0 : blockIdx.y * warps + warp, stride = SOLO ? 1 : gridDim.y * warps;
  for (int base = first * 256; base < H; base += stride * 256) {
    const Cols<U> c(base, lane, 32);
    V8 x = zero8(), acc = zero8();
    if (DOT) {
      Raw8<TR> xr;
      load8<U>(dot + t * ld_dot, c, H, xr);
      x = unpack(xr);
    }
#pragma unroll
    for (int b = 0; b < NK / B; ++b) {
      if (b * B >= k) break;
      Raw8<TR> v[B];
#pragma unroll
      for (int u = 0; u < B; ++u) {
        const int j = b * B + u;
        const int64_t s = j < k ? sh.at[j] : -1;
        if (s >= 0)
          load8<U>(rows + s, c, H, v[u]);
        else
          raw_zero(v[u]);
      }
#pragma unroll
      for (int u = 0; u < B; ++u) {
        const int j = b * B + u;
        if (j >= k || sh.at[j] < 0) continue;
        const V8 y = unpack(v[u]);
        acc = fma8(y, sh.w[j], acc);
        if (DOT) {
          float2 p = splat(0.f);
          dot8(x, y, p);
          part[DOT ? j / 8 : 0][j % 8] += p.x + p.y;
        }
      }
    }
    if (add != nullptr) {
      Raw8<TO> ar;
      load8<U>(add + t * ld_add, c, H, ar);
      acc = acc + unpack(ar);
    }
    store8<U>(out + t * ld_out, c, H, acc);
  }
  if (DOT) write_dw<SOLO, DOT ? NK / 8 : 1>(part, red, sh, dw + r0, k, warp, warps, tid);
}

// Warps that keep the memory busy, over the whole GPU.  28 fit on an SM with
// one per token (launch bounds: 4,096 tokens are then one wave; with five CTAs
// instead of seven dispatch's gradient took 73 us there, not 52).  Spread
// without dw waits for one load and then only stores: it wants more (4,096
// tokens: 47 us with 24 warps per SM, 36 with 120).
inline int warps_wanted() { return 24 * sm_count(); }

// Routes of a DOT kernel with half the registers for its sums.  Kernels without
// them have one form.
template <bool DOT>
constexpr int kFew = DOT ? 16 : kMaxK;

template <typename TT, typename TR, int U, bool DOT>
cudaError_t spread(const Rows& tok, const Rows& dot, const int32_t* slot_of, const float* w, int T, int k, int H,
                   int R, const Rows& out, float* dw, int32_t* status, cudaStream_t st) {
  const int pieces = (H + 255) / 256, want = DOT ? warps_wanted() : 5 * warps_wanted();
  // few tokens: more warps per token, then a token's routes over several CTAs
  const int warps = std::min({kMaxWarps, pieces, (want + T - 1) / T});
  const int64_t all = static_cast<int64_t>(T) * pieces;
  const int split = static_cast<int>(std::min<int64_t>(k, std::max<int64_t>(1, want / all)));
  const int jb = (k + split - 1) / split;
  auto go = [&](auto kern, dim3 grid, int threads) {
    return launch_pdl(kern, grid, dim3(threads), 0, st, static_cast<const TT*>(tok.p), tok.ld,
                      static_cast<const TR*>(dot.p), dot.ld, slot_of, w, T, k, jb, H, R, static_cast<TR*>(out.p),
                      out.ld, dw, status);
  };
  if (warps == 1 && split == 1) {
    const dim3 grid((T + kSoloWarps - 1) / kSoloWarps);
    return DOT && k <= 16 ? go(spread_kernel<TT, TR, U, DOT, kFew<DOT>, true>, grid, kSoloWarps * 32)
                          : go(spread_kernel<TT, TR, U, DOT, kMaxK, true>, grid, kSoloWarps * 32);
  }
  const dim3 grid(T, (k + jb - 1) / jb);
  return DOT && jb <= 16 ? go(spread_kernel<TT, TR, U, DOT, kFew<DOT>, false>, grid, warps * 32)
                         : go(spread_kernel<TT, TR, U, DOT, kMaxK, false>, grid, warps * 32);
}

template <typename TR, typename TO, int U, bool DOT>
cudaError_t join(const Rows& rows, const Rows& dot, const int32_t* slot_of, const float* w, int T, int k, int H, int R,
                 const Rows& out, const Rows& add, float* dw, int32_t* status, cudaStream_t st) {
  const int pieces = (H + 255) / 256;
  // few tokens: more warps per token, without dw on SMs of their own
  int warps = std::min({kMaxWarps, pieces, (warps_wanted() + T - 1) / T});
  int parts = 1;
  if (!DOT && warps > 1 && T < 4 * sm_count()) {
    warps = 1;
    parts = pieces;
  }
  auto go = [&](auto kern, dim3 grid, int threads) {
    return launch_pdl(kern, grid, dim3(threads), 0, st, static_cast<const TR*>(rows.p), rows.ld,
                      static_cast<const TR*>(dot.p), dot.ld, slot_of, w, T, k, H, R, static_cast<TO*>(out.p), out.ld,
                      static_cast<const TO*>(add.p), add.ld, dw, status);
  };
  if (warps == 1 && parts == 1) {
    const dim3 grid((T + kSoloWarps - 1) / kSoloWarps);
    return DOT && k <= 16 ? go(join_kernel<TR, TO, U, DOT, kFew<DOT>, true>, grid, kSoloWarps * 32)
                          : go(join_kernel<TR, TO, U, DOT, kMaxK, true>, grid, kSoloWarps * 32);
  }
  const dim3 grid(T, parts);
  return DOT && k <= 16 ? go(join_kernel<TR, TO, U, DOT, kFew<DOT>, false>, grid, warps * 32)
                        : go(join_kernel<TR, TO, U, DOT, kMaxK, false>, grid, warps * 32);
}

// f(type tag of a, type tag of b, the unit as an integral constant)
template <typename F>
cudaError_t by_types(int a, int b, int unit, F&& f) {
  auto g = [&](auto ta, auto tb) {
    if (unit == 8) return f(ta, tb, std::integral_constant<int, 8>());
    if (unit == 2) return f(ta, tb, std::integral_constant<int, 2>());
    return f(ta, tb, std::integral_constant<int, 1>());
  };
  if (a == MOE_ROW_F32) return b == MOE_ROW_F32 ? g(float(), float()) : g(float(), bf16_t());
  return b == MOE_ROW_F32 ? g(bf16_t(), float()) : g(bf16_t(), bf16_t());
}

}  // namespace

cudaError_t launch_spread(const Rows& tok, const Rows& dot, const int32_t* slot_of, const float* w, int T, int k,
                          int H, int R, const Rows& out, float* dw, int32_t* status, cudaStream_t st) {
  return by_types(tok.type, out.type, row_unit({tok, out, dot}), [&](auto tt, auto tr, auto u) {
    using TT = decltype(tt);
    using TR = decltype(tr);
    constexpr int U = decltype(u)::value;
    return dw != nullptr ? spread<TT, TR, U, true>(tok, dot, slot_of, w, T, k, H, R, out, dw, status, st)
                         : spread<TT, TR, U, false>(tok, dot, slot_of, w, T, k, H, R, out, dw, status, st);
  });
}

cudaError_t launch_join(const Rows& rows, const Rows& dot, const int32_t* slot_of, const float* w, int T, int k,
                        int H, int R, const Rows& out, const Rows& add, float* dw, int32_t* status, cudaStream_t st) {
  return by_types(rows.type, out.type, row_unit({rows, out, add, dot}), [&](auto tr, auto to, auto u) {
    using TR = decltype(tr);
    using TO = decltype(to);
    constexpr int U = decltype(u)::value;
    return dw != nullptr ? join<TR, TO, U, true>(rows, dot, slot_of, w, T, k, H, R, out, add, dw, status, st)
                         : join<TR, TO, U, false>(rows, dot, slot_of, w, T, k, H, R, out, add, dw, status, st);
  });
}

}  // namespace blk
}  // namespace moe
