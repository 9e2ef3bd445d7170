// Gradient of the renormalised top-k router.
//
// The weights are the softmax over a token's k selected logits, so
//   dl_j = w_j (dw_j - sum_i w_i dw_i),
// the gradient of x is the dl-weighted sum of k router rows (the join of
// dispatch.cu, with the router as its rows and the expert IDs as its slots)
// and that of the router sums dl x over the routes of each expert, which the
// grouping has put side by side.
//
// A sparse sum, not a matrix product over all experts: k of E logits carry a
// gradient, so the dense form computes E / k times the work (and would have
// to hold dl in bf16 to use the tensor cores).  Bound by L2: x and the router
// stay there, and each of their rows is read once per route.
//
// An expert's routes are cut into units of at most kUnit, so that a popular
// expert is shared by many CTAs; an expert of one unit is written directly,
// the units of others leave partial rows that a last launch adds in order.
#include <algorithm>

#include "launch.h"
#include "rows.cuh"

namespace moe {
namespace blk {

namespace {

constexpr int kUnit = 256;         // routes per unit
constexpr int kPlanThreads = 1024;  // >= kMaxE
constexpr int kBatch = 8;          // rows whose loads a thread has in flight
constexpr int kMaxSlab = 256;      // threads per CTA, eight columns each

// Workspace (int32 unless said): [E+1] first unit of each expert, [E] first
// partial row of each expert, [1] whether the offsets are bad, then, 256-byte
// aligned, the partial rows [max_partials][H] f32 and their bias sums
// [max_partials] f32.
__host__ __device__ inline int max_partials(int R) { return 2 * (R / kUnit) + 1; }
struct Ws {
  int32_t *unit0, *part0, *bad;
  float *rows, *bias;
};
__host__ __device__ inline Ws ws_layout(void* p, int R, int E, int H) {
  Ws w;
  w.unit0 = static_cast<int32_t*>(p);
  w.part0 = w.unit0 + E + 1;
  w.bad = w.part0 + E;
  const size_t head = (static_cast<size_t>(2 * E + 2) * 4 + 255) / 256 * 256;
  w.rows = reinterpret_cast<float*>(static_cast<char*>(p) + head);
  w.bias = w.rows + static_cast<size_t>(max_partials(R)) * H;
  return w;
}

__device__ __forceinline__ int block_scan_excl(int v, int* warp_tot) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += y;
  }
  if (lane == 31) warp_tot[warp] = incl;
  __syncthreads();
  int before = 0;
  for (int i = 0; i < warp; ++i) before += warp_tot[i];
  __syncthreads();
  return before + incl - v;
}

// CTA 0: the units of every expert.  The others: dl, one warp per token.
__global__ void __launch_bounds__(kPlanThreads)
    route_plan_kernel(const float* __restrict__ dw, const float* __restrict__ w, const int32_t* __restrict__ offsets,
                      int T, int k, int E, int H, float* __restrict__ dl, void* ws, int plan, int32_t* status) {
  __shared__ int warp_tot[32];
  __shared__ int bad;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31;
  if (blockIdx.x == 0) {
    if (!plan) return;
    const int R = T * k;
    const Ws s = ws_layout(ws, R, E, H);
    if (tid == 0) bad = 0;
    __syncthreads();
    int n = 0;
    if (tid < E && R > 0) {  // no routes: the grouping wrote no offsets
      const int a = offsets[tid], b = offsets[tid + 1];
      if (a < 0 || b < a || b > R || (tid == 0 && a != 0) || (tid == E - 1 && b != R)) bad = 1;
      n = b - a;
    }
    __syncthreads();
    const int units = tid < E && !bad ? max(1, (n + kUnit - 1) / kUnit) : 0;
    const int u0 = block_scan_excl(units, warp_tot);
    const int p0 = block_scan_excl(units > 1 ? units : 0, warp_tot);
    if (tid < E) {
      s.unit0[tid] = u0;
      s.part0[tid] = p0;
      if (tid == E - 1) s.unit0[E] = u0 + units;
    }
    if (tid == 0) {
      *s.bad = bad;
      if (bad) set_status(status, MOE_DEV_BAD_EXPERT);
    }
    return;
  }
  const int warps = kPlanThreads / 32;
  for (int64_t t = static_cast<int64_t>(blockIdx.x - 1) * warps + (tid >> 5); t < T;
       t += static_cast<int64_t>(gridDim.x - 1) * warps) {
    const float wj = lane < k ? w[t * k + lane] : 0.f;
    const float gj = lane < k ? dw[t * k + lane] : 0.f;
    float m = lane < k ? wj * gj : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
    if (lane < k) dl[t * k + lane] = wj * (gj - m);
  }
}

// grid (unit, slab of 8 * blockDim.x columns)
template <bool VEC>
__global__ void __launch_bounds__(kMaxSlab)
    route_rows_kernel(const float* __restrict__ dl, const int32_t* __restrict__ offsets,
                      const int32_t* __restrict__ perm, const bf16_t* __restrict__ x, int64_t ldx, int T, int k, int E,
                      int H, float* dwr, int64_t ld_dw, float* dbias, void* ws, int32_t* status) {
  __shared__ int expert;
  __shared__ int tok[kUnit];
  __shared__ float g[kUnit];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  const int R = T * k;
  const Ws s = ws_layout(ws, R, E, H);
  if (*s.bad) return;
  const int u = blockIdx.x;
  if (tid == 0) expert = -1;
  __syncthreads();
  for (int e = tid; e < E; e += blockDim.x)
    if (s.unit0[e] <= u && u < s.unit0[e + 1]) expert = e;
  __syncthreads();
  const int e = expert;
  if (e < 0) return;
  const int part = u - s.unit0[e];
  const bool direct = s.unit0[e + 1] - s.unit0[e] == 1;
  const int a = R > 0 ? offsets[e] + part * kUnit : 0;
  const int n = R > 0 ? min(kUnit, offsets[e + 1] - a) : 0;
  for (int i = tid; i < n; i += blockDim.x) {
    const int r = perm[a + i];
    const bool ok = r >= 0 && r < R;
    if (!ok) set_status(status, MOE_DEV_BAD_EXPERT);
    tok[i] = ok ? r / k : -1;
    g[i] = ok ? dl[r] : 0.f;
  }
  __syncthreads();
  if (dbias != nullptr && blockIdx.y == 0 && tid < 32) {
    float b = 0.f;
    for (int i = tid; i < n; i += 32) b += g[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) b += __shfl_xor_sync(0xffffffffu, b, o);
    if (tid == 0) (direct ? dbias[e] : s.bias[s.part0[e] + part]) = b;
  }
  if (dwr == nullptr) return;
  const Cols<VEC> c(blockIdx.y * blockDim.x * 8, tid, blockDim.x);
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
  for (int i0 = 0; i0 < n; i0 += kBatch) {
    Raw8<bf16_t> v[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int t = i0 + b < n ? tok[i0 + b] : -1;
      if (t >= 0)
        load8<VEC>(x + t * ldx, c, H, v[b]);
      else
        raw_zero(v[b]);
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (i0 + b >= n || tok[i0 + b] < 0) continue;
      float f[8];
      unpack(v[b], f);
      const float w = g[i0 + b];
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = fmaf(w, f[i], acc[i]);
    }
  }
  if (direct)
    store8<VEC>(dwr + e * ld_dw, c, H, acc);
  else
    // partial rows are packed [H]: whole vectors only where H allows it
    for (int i = 0; i < 8; ++i)
      if (c.first + i * c.step < H)
        s.rows[static_cast<size_t>(s.part0[e] + part) * H + c.first + i * c.step] = acc[i];
}

// grid (expert, 256 columns): the experts of several units.
__global__ void __launch_bounds__(256) route_join_kernel(int T, int k, int E, int H, float* dwr, int64_t ld_dw,
                                                         float* dbias, void* ws) {
  pdl_wait();
  pdl_trigger();
  const Ws s = ws_layout(ws, T * k, E, H);
  if (*s.bad) return;
  const int e = blockIdx.x;
  const int n = s.unit0[e + 1] - s.unit0[e];
  if (n <= 1) return;
  const int p0 = s.part0[e];
  const int col = blockIdx.y * 256 + threadIdx.x;
  if (dwr != nullptr && col < H) {
    float a = 0.f;
    for (int p = 0; p < n; ++p) a += s.rows[static_cast<size_t>(p0 + p) * H + col];
    dwr[e * ld_dw + col] = a;
  }
  if (dbias != nullptr && blockIdx.y == 0 && threadIdx.x == 0) {
    float b = 0.f;
    for (int p = 0; p < n; ++p) b += s.bias[p0 + p];
    dbias[e] = b;
  }
}

}  // namespace

size_t route_grad_ws_bytes(int T, int k, int E, int H) {
  const int R = T * k;
  const size_t head = (static_cast<size_t>(2 * E + 2) * 4 + 255) / 256 * 256;
  return (head + static_cast<size_t>(max_partials(R)) * (H + 1) * sizeof(float) + 255) / 256 * 256;
}

cudaError_t launch_route_grad(const RouteGradArgs& a, cudaStream_t st) {
  const int R = a.T * a.k;
  const int plan = a.dw_router.p != nullptr || a.dbias != nullptr;
  const int warps = kPlanThreads / 32;
  const int dl_ctas = std::min((a.T + warps - 1) / warps, 4 * sm_count());
  cudaError_t e = cudaSuccess;
  if (plan || dl_ctas > 0) {
    e = launch_pdl(route_plan_kernel, dim3(1 + dl_ctas), dim3(kPlanThreads), 0, st, a.dw, a.w, a.offsets, a.T, a.k,
                   a.E, a.H, a.dlogits, a.ws, plan, a.status);
    if (e != cudaSuccess) return e;
  }
  if (a.dx.p != nullptr && a.T > 0) {
    const Rows none = {nullptr, 0, MOE_ROW_BF16};
    e = launch_join(a.w_router, none, a.ids, a.dlogits, a.T, a.k, a.H, a.E, a.dx, a.add, nullptr, a.status, st);
    if (e != cudaSuccess) return e;
  }
  if (!plan) return cudaSuccess;
  const int chunks = (a.H + 7) / 8;
  const int slabs = a.dw_router.p != nullptr ? (chunks + kMaxSlab - 1) / kMaxSlab : 1;
  const int nt = a.dw_router.p != nullptr ? ((chunks + slabs - 1) / slabs + 31) / 32 * 32 : 128;
  const int units = a.E + R / kUnit;
  const bool vec = vec_ok(a.x) && vec_ok(a.dw_router);
  auto go = [&](auto kern) {
    return launch_pdl(kern, dim3(units, slabs), dim3(nt), 0, st, a.dlogits, a.offsets, a.perm,
                      static_cast<const bf16_t*>(a.x.p), a.x.ld, a.T, a.k, a.E, a.H,
                      static_cast<float*>(a.dw_router.p), a.dw_router.ld, a.dbias, a.ws, a.status);
  };
  e = vec ? go(route_rows_kernel<true>) : go(route_rows_kernel<false>);
  if (e != cudaSuccess || R <= kUnit) return e;
  return launch_pdl(route_join_kernel, dim3(a.E, (a.H + 255) / 256), dim3(256), 0, st, a.T, a.k, a.E, a.H,
                    static_cast<float*>(a.dw_router.p), a.dw_router.ld, a.dbias, a.ws);
}

}  // namespace blk
}  // namespace moe
