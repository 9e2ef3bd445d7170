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
constexpr int kRowThreads = 256;   // threads per CTA of the row sums

// A unit: n routes of expert e from slot s0 on; part is where its partial row
// goes, or -1 where it is the expert's only unit and writes the result.
struct Unit {
  int32_t e, s0, n, part;
};

// Workspace, each part 256-byte aligned: the units, each expert's first
// partial row and how many it has ({first, count}, count 0: written
// directly), partial rows [..][H] f32, their bias sums f32.
__host__ __device__ inline int max_units(int R, int E) { return E + R / kUnit; }
__host__ __device__ inline int max_partials(int R) { return 2 * (R / kUnit) + 1; }
__host__ __device__ inline size_t round256(size_t n) { return (n + 255) / 256 * 256; }
struct Ws {
  Unit* units;
  int2* parts;
  float *rows, *bias;
  size_t bytes;
};
__host__ __device__ inline Ws ws_layout(void* p, int R, int E, int H) {
  char* c = static_cast<char*>(p);
  size_t at = 0;
  Ws w;
  w.units = reinterpret_cast<Unit*>(c + at);
  at += round256(sizeof(Unit) * max_units(R, E));
  w.parts = reinterpret_cast<int2*>(c + at);
  at += round256(sizeof(int2) * E);
  w.rows = reinterpret_cast<float*>(c + at);
  at += round256(sizeof(float) * static_cast<size_t>(max_partials(R)) * H);
  w.bias = reinterpret_cast<float*>(c + at);
  w.bytes = at + round256(sizeof(float) * max_partials(R));
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
  __shared__ int first[kPlanThreads], start[kPlanThreads], count[kPlanThreads], part0[kPlanThreads];
  __shared__ int bad, total;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31;
  if (blockIdx.x == 0) {
    if (!plan) return;
    const int R = T * k;
    const Ws s = ws_layout(ws, R, E, H);
    if (tid == 0) bad = 0;
    __syncthreads();
    int n = 0, a = 0;
    if (tid < E && R > 0) {  // no routes: the grouping wrote no offsets
      a = offsets[tid];
      const int b = offsets[tid + 1];
      if (a < 0 || b < a || b > R || (tid == 0 && a != 0) || (tid == E - 1 && b != R)) bad = 1;
      n = b - a;
    }
    __syncthreads();
    // bad offsets: every unit is marked as none
    const int units = tid < E && !bad ? max(1, (n + kUnit - 1) / kUnit) : 0;
    const int p0 = block_scan_excl(units > 1 ? units : 0, warp_tot);
    first[tid] = block_scan_excl(units, warp_tot);
    start[tid] = a;
    count[tid] = n;
    part0[tid] = units > 1 ? p0 : -1;
    if (tid < E) s.parts[tid] = make_int2(p0, units > 1 ? units : 0);
    if (tid == kPlanThreads - 1) total = first[tid] + units;
    __syncthreads();
    for (int u = tid; u < max_units(R, E); u += kPlanThreads) {
      Unit d = {-1, 0, 0, -1};
      if (u < total) {
        int lo = 0, hi = E;  // the expert whose first unit is the last at or before u
        while (hi - lo > 1) {
          const int mid = (lo + hi) / 2;
          if (first[mid] <= u)
            lo = mid;
          else
            hi = mid;
        }
        const int i = u - first[lo];
        d = {lo, start[lo] + i * kUnit, min(kUnit, count[lo] - i * kUnit), part0[lo] < 0 ? -1 : part0[lo] + i};
      }
      s.units[u] = d;
    }
    if (tid == 0 && bad) set_status(status, MOE_DEV_BAD_EXPERT);
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

// grid (unit, slab of 8 cw columns).  The CTA's threads are cw columns of
// eight by kRowThreads / cw row groups; a row group sums every such route of
// the unit, and the first adds the others in order.
template <bool VEC>
__global__ void __launch_bounds__(kRowThreads)
    route_rows_kernel(const float* __restrict__ dl, const int32_t* __restrict__ perm, const bf16_t* __restrict__ x,
                      int64_t ldx, int T, int k, int E, int H, int cw, float* dwr, int64_t ld_dw, float* dbias,
                      void* ws, int32_t* status) {
  __shared__ int2 route[kUnit];  // token (-1: none) and the bits of dl
  __shared__ float red[kRowThreads * 8];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  const int R = T * k;
  const Ws s = ws_layout(ws, R, E, H);
  const Unit un = s.units[blockIdx.x];
  if (un.e < 0) return;
  const int n = un.n;
  for (int i = tid; i < n; i += kRowThreads) {
    const int r = perm[un.s0 + i];
    const bool ok = r >= 0 && r < R;
    if (!ok) set_status(status, MOE_DEV_BAD_EXPERT);
    route[i] = make_int2(ok ? r / k : -1, ok ? __float_as_int(dl[r]) : 0);
  }
  __syncthreads();
  if (dbias != nullptr && blockIdx.y == 0 && tid < 32) {
    float b = 0.f;
    for (int i = tid; i < n; i += 32) b += __int_as_float(route[i].y);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) b += __shfl_xor_sync(0xffffffffu, b, o);
    if (tid == 0) (un.part < 0 ? dbias[un.e] : s.bias[un.part]) = b;
  }
  if (dwr == nullptr) return;
  const int rg = kRowThreads / cw, g = tid / cw, col = tid - g * cw;
  const Cols<VEC> c(blockIdx.y * cw * 8, col, cw);
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
  for (int i0 = g; i0 < n; i0 += kBatch * rg) {
    Raw8<bf16_t> v[kBatch];
    float w[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int i = i0 + b * rg;
      const int2 rt = i < n ? route[i] : make_int2(-1, 0);
      w[b] = __int_as_float(rt.y);
      if (rt.x >= 0)
        load8<VEC>(x + rt.x * ldx, c, H, v[b]);
      else
        raw_zero(v[b]);
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      float f[8];
      unpack(v[b], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = fmaf(w[b], f[i], acc[i]);
    }
  }
  if (rg > 1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) red[i * kRowThreads + tid] = acc[i];
    __syncthreads();
    if (g > 0) return;
    for (int o = 1; o < rg; ++o)
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += red[i * kRowThreads + o * cw + col];
  }
  if (un.part < 0) {
    store8<VEC>(dwr + un.e * ld_dw, c, H, acc);
  } else {
    float* out = s.rows + static_cast<size_t>(un.part) * H;  // packed: whole vectors only where H allows it
    if (VEC && H % 8 == 0) {
      store8<VEC>(out, c, H, acc);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c.first + i * c.step < H) out[c.first + i * c.step] = acc[i];
    }
  }
}

// grid (expert, 256 columns): the experts of several units.
__global__ void __launch_bounds__(256) route_join_kernel(int T, int k, int E, int H, float* dwr, int64_t ld_dw,
                                                         float* dbias, void* ws) {
  pdl_wait();
  pdl_trigger();
  const Ws s = ws_layout(ws, T * k, E, H);
  const int e = blockIdx.x;
  const int p0 = s.parts[e].x, n = s.parts[e].y;
  if (n == 0) return;
  const int col = blockIdx.y * 256 + threadIdx.x;
  if (dwr != nullptr && col < H) {
    float a = 0.f;
#pragma unroll 4
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
  return ws_layout(nullptr, T * k, E, H).bytes;
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
  // 64 columns of eight by 4 row groups; narrower rows: fewer columns
  const int chunks = (a.H + 7) / 8;
  const int cw = chunks > 32 ? 64 : chunks > 16 ? 32 : 16;
  const int slabs = a.dw_router.p != nullptr ? (chunks + cw - 1) / cw : 1;
  const bool vec = vec_ok(a.x) && vec_ok(a.dw_router);
  auto go = [&](auto kern) {
    return launch_pdl(kern, dim3(max_units(R, a.E), slabs), dim3(kRowThreads), 0, st, a.dlogits, a.perm,
                      static_cast<const bf16_t*>(a.x.p), a.x.ld, a.T, a.k, a.E, a.H, cw,
                      static_cast<float*>(a.dw_router.p), a.dw_router.ld, a.dbias, a.ws, a.status);
  };
  e = vec ? go(route_rows_kernel<true>) : go(route_rows_kernel<false>);
  if (e != cudaSuccess || R <= kUnit) return e;
  return launch_pdl(route_join_kernel, dim3(a.E, (a.H + 255) / 256), dim3(256), 0, st, a.T, a.k, a.E, a.H,
                    static_cast<float*>(a.dw_router.p), a.dw_router.ld, a.dbias, a.ws);
}

}  // namespace blk
}  // namespace moe
