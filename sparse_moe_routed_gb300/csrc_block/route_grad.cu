// Gradient of the renormalised top-k router.
//
// The weights are the softmax over a token's k selected logits, so
//   dl_j = w_j (dw_j - sum_i w_i dw_i),
// the gradient of x is the dl-weighted sum of k router rows, and that of the
// router sums dl x over the routes of each expert, which the grouping has put
// side by side.
//
// Sparse sums, not matrix products over all experts: x and the router stay in
// L2, and what bounds both sums is reading each of their rows once per route
// through the SMs, T k H elements each whatever E is.  There is no dense form.
// On the tensor cores, with dl in three bf16 terms (fp32's 24 bits), it would
// take 12 T E H operations, which at the measured bf16 rate are 35 us for
// 4,096 tokens of width 2,560 and 512 experts, 9 for 128 and 4 for 64; the
// sparse sums take 49 to 57 us for 64 to 512 experts with top 10 and even
// popularity.  So they are the right form where E / k is large, and leave time
// on the table where it is small.
//
// dx: with many tokens a CTA keeps a slab of the router's columns in shared
// memory and reads every route's row from there; with few, or rows that are
// not aligned, it is the join of dispatch.cu with the router as its rows and
// the expert IDs as its slots.
// dw_router: one warp per unit of some routes of one expert and 256 columns.  An
// expert of one unit is written directly; the units of a popular expert leave
// partial rows that a last launch adds in order.
#include <algorithm>

#include "norm.h"
#include "stage.cuh"

namespace moe {
namespace blk {

namespace {

// Routes per unit: short units keep few routes from waiting on one warp's
// long chain, long ones save partial rows.  Per call with dx NULL, top 10 of
// 512 experts, width 2,560, popularity 1 / rank: 512 tokens 13.7 us with units
// of 64, 13.8 with 32, 16.0 with 128; 1,024 tokens 16.9 with 64, 19.2 with 128;
// 4,096 tokens 36.2 with 128, 39.3 with 64, 39.9 with 256; 16,384 tokens 95
// with 256, 120 with 128.  Not tuned for other experts or widths: few experts
// of narrow rows get few warps (8 experts, 16,384 routes, 256 columns: 128 warps,
// and the call takes 30 us for a floor of 3).
inline int unit_for(int R) { return R <= 16000 ? 64 : R <= 100000 ? 128 : 256; }
constexpr int kPlanThreads = 1024;  // >= kMaxE
// Rows whose loads a thread has in flight (single elements need eight registers
// a row: the call on odd rows 134 us with four, 166 with eight at 4,096 tokens).
template <int U>
constexpr int kBatch = U == 1 ? 4 : 8;
constexpr int kRowWarps = 4;        // warps per CTA of the row sums

// A unit: n routes of expert e (-1: no unit) from slot s0 on; part is where
// its partial row goes, or -1 where it is the expert's only unit and writes
// the result.
struct Unit {
  int32_t e, s0, n, part;
};

// An expert of n > 1 units (0: none): partial rows part0 .. part0 + n - 1.
struct Multi {
  int32_t e, part0, n, pad;
};

// With unit u an expert of n routes has ceil(n / u) <= n / u + 1 units, and one
// of several has n > u routes: at most R / u experts, and no more than E.
inline int max_units(int R, int E) { return E + R / unit_for(R); }
inline int max_multi(int R, int E) { return std::min(E, R / unit_for(R)); }
inline int max_partials(int R, int E) { return R / unit_for(R) + max_multi(R, E) + 1; }

// The workspace's parts, 256-byte aligned: the units, the experts of several
// units, partial rows [..][H], their bias sums.
struct Ws {
  Unit* units;
  Multi* multi;
  float *rows, *bias;
  size_t bytes;
};
Ws ws_layout(void* p, int R, int E, int H) {
  char* c = static_cast<char*>(p);
  size_t at = 0;
  auto take = [&](size_t n) {
    char* q = c + at;
    at += (n + 255) / 256 * 256;
    return q;
  };
  Ws w;
  w.units = reinterpret_cast<Unit*>(take(sizeof(Unit) * max_units(R, E)));
  w.multi = reinterpret_cast<Multi*>(take(sizeof(Multi) * max_multi(R, E)));
  w.rows = reinterpret_cast<float*>(take(sizeof(float) * static_cast<size_t>(max_partials(R, E)) * H));
  w.bias = reinterpret_cast<float*>(take(sizeof(float) * max_partials(R, E)));
  w.bytes = at;
  return w;
}

// Up to this many tokens an expert is one unit (n <= T where a token's experts
// are distinct): no plan and no join (16 tokens, top 4 of 64 experts: 5.4 us
// against 7.8; at 128 tokens one warp's chain costs more, 13.8 against 12.8).
constexpr int kDirectTokens = 64;

// Do a thread's offsets rise from 0 to R?
__device__ __forceinline__ bool offsets_bad(const int32_t* offsets, int e, int E, int R, int& a, int& n) {
  a = offsets[e];
  const int b = offsets[e + 1];
  n = b - a;
  return a < 0 || b < a || b > R || (e == 0 && a != 0) || (e == E - 1 && b != R);
}

// Exclusive sum over the CTA's threads; returns the total in `total`.
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t* warp_tot, uint64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t incl = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += y;
  }
  if (lane == 31) warp_tot[warp] = incl;
  __syncthreads();
  uint64_t before = lane < warp ? warp_tot[lane] : 0, all = warp_tot[lane];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, o);
    all += __shfl_xor_sync(0xffffffffu, all, o);
  }
  total = all;
  return before + incl - v;
}

// dl (and a look at the expert IDs), one warp per token, and with `plan` CTA 0
// the units of every expert.
__global__ void __launch_bounds__(kPlanThreads)
    route_plan_kernel(const float* __restrict__ dw, const float* __restrict__ w, const int32_t* __restrict__ ids,
                      const int32_t* __restrict__ offsets, int T, int k, int E, float* __restrict__ dl,
                      Unit* units_out, Multi* multi_out, int units_max, int multi_max, int plan, int unit,
                      int32_t* status) {
  __shared__ uint64_t warp_tot[32];
  __shared__ int start[kPlanThreads], count[kPlanThreads], part0[kPlanThreads];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31;
  if (plan && blockIdx.x == 0) {
    int n = 0, a = 0;
    const bool bad = __syncthreads_or(tid < E && offsets_bad(offsets, tid, E, T * k, a, n)) != 0;
    // bad offsets: no unit at all.  One sum of three: units (26 bits), partial
    // rows (27), experts of several units (11).
    const int units = tid < E && !bad ? max(1, (n + unit - 1) / unit) : 0;
    const bool several = units > 1;
    uint64_t total;
    const uint64_t at = block_scan(static_cast<uint64_t>(units) |
                                       (several ? static_cast<uint64_t>(units) << 26 | 1ull << 53 : 0ull),
                                   warp_tot, total);
    const int p0 = static_cast<int>(at >> 26 & 0x7ffffff), m0 = static_cast<int>(at >> 53);
    const int all = static_cast<int>(total & 0x3ffffff), shared = static_cast<int>(total >> 26 & 0x7ffffff);
    // the units of experts with several come first: they are the long ones,
    // and what starts last should be short
    part0[tid] = p0;
    start[tid] = a;
    count[tid] = n;
    if (several)
      multi_out[m0] = {tid, p0, units, 0};
    else if (units == 1)
      units_out[shared + static_cast<int>(at & 0x3ffffff) - p0] = {tid, a, n, -1};
    for (int i = static_cast<int>(total >> 53) + tid; i < multi_max; i += kPlanThreads) multi_out[i] = {0, 0, 0, 0};
    for (int u = all + tid; u < units_max; u += kPlanThreads) units_out[u] = {-1, 0, 0, -1};
    __syncthreads();
    for (int u = tid; u < shared; u += kPlanThreads) {
      int lo = 0, hi = E;  // the last expert whose first partial row is at or before u
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (part0[mid] <= u)
          lo = mid;
        else
          hi = mid;
      }
      const int i = u - part0[lo];
      units_out[u] = {lo, start[lo] + i * unit, min(unit, count[lo] - i * unit), u};
    }
    if (tid == 0 && bad) set_status(status, MOE_DEV_BAD_EXPERT);
    return;
  }
  const int warps = kPlanThreads / 32;
  for (int64_t t = static_cast<int64_t>(blockIdx.x - plan) * warps + (tid >> 5); t < T;
       t += static_cast<int64_t>(gridDim.x - plan) * warps) {
    const float wj = lane < k ? w[t * k + lane] : 0.f;
    const float gj = lane < k ? dw[t * k + lane] : 0.f;
    if (lane < k) {
      const int e = ids[t * k + lane];
      if (e < 0 || e >= E) set_status(status, MOE_DEV_BAD_EXPERT);
    }
    float m = lane < k ? wj * gj : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
    if (lane < k) dl[t * k + lane] = wj * (gj - m);
  }
}

// One warp per unit and piece of 256 columns: it needs no other, so that the
// chain of loads in front of its rows (unit, route, dl) overlaps the rows of
// the SM's other warps.  grid (units / kRowWarps, pieces).  DIRECT: the units
// are the experts.
template <int U, bool DIRECT>
__global__ void __launch_bounds__(kRowWarps * 32)
    route_rows_kernel(const float* __restrict__ dl, const int32_t* __restrict__ offsets,
                      const int32_t* __restrict__ perm, const bf16_t* __restrict__ x, int64_t ldx, int R, int k, int E,
                      int H, const Unit* units, int units_max, float* dwr, int64_t ld_dw, float* dbias,
                      float* part_rows, float* part_bias, int32_t* status) {
  __shared__ int2 routes[kRowWarps][32];  // token (-1: none) and the bits of dl
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int unit = blockIdx.x * kRowWarps + warp;
  Unit un = {-1, 0, 0, -1};
  if (DIRECT) {
    int a = 0, n = 0;
    bool bad = false;
    if (R > 0)  // no routes: the grouping wrote no offsets
      for (int e = threadIdx.x; e < E; e += kRowWarps * 32) bad |= offsets_bad(offsets, e, E, R, a, n);
    if (__syncthreads_or(bad)) {
      if (threadIdx.x == 0) set_status(status, MOE_DEV_BAD_EXPERT);
      return;
    }
    if (unit < E) {
      const int s0 = R > 0 ? offsets[unit] : 0;
      un = {unit, s0, R > 0 ? offsets[unit + 1] - s0 : 0, -1};
    }
  } else if (unit < units_max) {
    un = units[unit];
  }
  if (un.e < 0) return;
  auto fetch = [&](int i) {
    if (i >= un.n) return make_int2(-1, 0);
    const int r = perm[un.s0 + i];
    if (r >= 0 && r < R) return make_int2(r / k, __float_as_int(dl[r]));
    set_status(status, MOE_DEV_BAD_EXPERT);
    return make_int2(-1, 0);
  };
  const Cols<U> c(blockIdx.y * 256, lane, 32);
  const bool whole = U == 8 && c.first + 8 <= H;
  V8 acc = zero8();
  float bias = 0.f;
  int2 next = fetch(lane);
  for (int i0 = 0; i0 < un.n; i0 += 32) {
    __syncwarp();
    routes[warp][lane] = next;
    bias += __int_as_float(next.y);
    const unsigned valid = __ballot_sync(0xffffffffu, next.x >= 0);
    __syncwarp();
    next = fetch(i0 + 32 + lane);
    if (dwr == nullptr) continue;
#pragma unroll 1
    for (int j0 = 0; j0 < 32 && valid >> j0 != 0; j0 += kBatch<U>) {
      Raw8<bf16_t> v[kBatch<U>];
      float w[kBatch<U>];
      if (whole && (~(valid >> j0) & ((1u << kBatch<U>) - 1)) == 0) {  // the usual batch: nothing to test per row
#pragma unroll
        for (int b = 0; b < kBatch<U>; ++b) {
          const int2 rt = routes[warp][j0 + b];
          w[b] = __int_as_float(rt.y);
          load_vec(x + rt.x * ldx + c.first, v[b]);
        }
      } else {
#pragma unroll
        for (int b = 0; b < kBatch<U>; ++b) {
          const int2 rt = routes[warp][j0 + b];
          w[b] = __int_as_float(rt.y);
          if (rt.x >= 0)
            load8<U>(x + rt.x * ldx, c, H, v[b]);
          else
            raw_zero(v[b]);
        }
      }
#pragma unroll
      for (int b = 0; b < kBatch<U>; ++b) acc = fma8(unpack(v[b]), w[b], acc);
    }
  }
  if (dbias != nullptr && blockIdx.y == 0) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) bias += __shfl_xor_sync(0xffffffffu, bias, o);
    if (lane == 0) (un.part < 0 ? dbias[un.e] : part_bias[un.part]) = bias;
  }
  if (dwr == nullptr) return;
  if (un.part < 0) {
    store8<U>(dwr + un.e * ld_dw, c, H, acc);
  } else {
    float* out = part_rows + static_cast<size_t>(un.part) * H;  // packed: whole vectors only where H allows it
    if (U == 8 && H % 8 == 0) {
      store8<U>(out, c, H, acc);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c.at(i) < H) out[c.at(i)] = el(acc, i);
    }
  }
}

// grid (expert of several units, 1,024 columns): the partial rows in order.
__global__ void __launch_bounds__(256) route_join_kernel(const Multi* multi, const float* rows, const float* bias,
                                                         int H, float* dwr, int64_t ld_dw, float* dbias) {
  pdl_wait();
  pdl_trigger();
  const Multi m = multi[blockIdx.x];
  if (m.n == 0) return;
  if (dwr != nullptr) {
    float a[4] = {0.f, 0.f, 0.f, 0.f};
    const int col = blockIdx.y * 1024 + threadIdx.x;
    const float* src = rows + static_cast<size_t>(m.part0) * H + col;
#pragma unroll 2
    for (int p = 0; p < m.n; ++p)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (col + i * 256 < H) a[i] += src[static_cast<size_t>(p) * H + i * 256];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (col + i * 256 < H) dwr[m.e * ld_dw + col + i * 256] = a[i];
  }
  if (dbias != nullptr && blockIdx.y == 0 && threadIdx.x == 0) {
    float b = 0.f;
    for (int p = 0; p < m.n; ++p) b += bias[m.part0 + p];
    dbias[m.e] = b;
  }
}

// dx with a slab of the router's columns in shared memory: CTA (slab, part of
// the tokens) copies its columns of all E rows once and then reads every
// route's row from there; row E is zeros, for routes that are none.  Sixteen
// lanes of eight columns work on a token, two tokens per warp.
constexpr int kSlabColumns = 128;
constexpr int kSlabThreads = 1024;
constexpr int kSlabBatch = 2;  // rows whose reads a thread has in flight (1, 4: 28.7 and 29.0 us, 2: 26.9)
// From this many elements of routed rows on (and where E + 1 rows of 128
// columns fit): 26.9 us against the join's 32.5 at 4,096 tokens, top 10 of 512
// experts, width 2,560, and 82 against 107 at 16,384; 17.3 against 18.5 at
// 2,048, but 14.8 against 13.2 at 2,048 with top 4 of 64.  Other numbers of
// experts were not measured.
constexpr int64_t kSlabElements = 50'000'000;

template <typename TO>
__global__ void __launch_bounds__(kSlabThreads)
    route_dx_kernel(const bf16_t* __restrict__ wr, int64_t ld_wr, const int32_t* __restrict__ ids,
                    const float* __restrict__ dl, int T, int k, int E, int H, TO* dx, int64_t ld_dx, const TO* add,
                    int64_t ld_add) {
  extern __shared__ __align__(16) unsigned char slab[];  // [E + 1][C] bf16
  constexpr int C = kSlabColumns, kLanes = C / 8, kTokens = 32 / kLanes;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int col = blockIdx.x * C;
  for (int i = tid; i < (E + 1) * kLanes; i += kSlabThreads) {
    const int e = i / kLanes, c = col + (i % kLanes) * 8;
    const int n = e < E ? max(0, min(8, H - c)) : 0;  // columns of the vector that exist; the rest become zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(slab)) + i * 16),
                 "l"(n > 0 ? wr + e * ld_wr + c : wr), "r"(n * 2)
                 : "memory");
  }
  copies_commit();
  copies_wait();
  __syncthreads();
  const int sub = lane / kLanes, l = lane % kLanes;
  const Cols<8> c(col, l, kLanes);
  const unsigned char* mine = slab + l * 16;
  const int64_t step = static_cast<int64_t>(gridDim.y) * (kSlabThreads / 32) * kTokens;
  // lane l of the token's lanes reads routes l, l + kLanes, ...
  auto route = [&](int64_t t, int j, int& id, float& g) {
    id = E;
    g = 0.f;
    if (t < T && j < k) {
      id = ids[t * k + j];
      g = dl[t * k + j];
      if (id < 0 || id >= E) id = E, g = 0.f;  // flagged where dl was computed
    }
  };
  int64_t t = (static_cast<int64_t>(blockIdx.y) * (kSlabThreads / 32) + warp) * kTokens + sub;
  // the next token's first routes and add are loaded while this one's rows are summed
  int id_next;
  float g_next;
  Raw8<TO> a_next;
  auto ahead = [&](int64_t at) {
    route(at, l, id_next, g_next);
    raw_zero(a_next);
    if (at < T && add != nullptr) load8<8>(add + at * ld_add, c, H, a_next);
  };
  ahead(t);
  for (; t - sub < T; t += step) {
    int id = id_next;
    float g = g_next;
    const Raw8<TO> ar = a_next;
    ahead(t + step);
    V8 acc = zero8();
    for (int j0 = 0;;) {
      id *= C * 2;  // bytes to the row
      const int n = min(kLanes, k - j0);
#pragma unroll 1
      for (int b = 0; b < n; b += kSlabBatch) {
        Raw8<bf16_t> q[kSlabBatch];
        float w[kSlabBatch];
#pragma unroll
        for (int u = 0; u < kSlabBatch; ++u) {
          // a place past k - j0 (and within the token's lanes) holds row E
          const uint4 row = *reinterpret_cast<const uint4*>(mine + __shfl_sync(0xffffffffu, id, b + u, kLanes));
          q[u].v[0] = row.x, q[u].v[1] = row.y, q[u].v[2] = row.z, q[u].v[3] = row.w;
          w[u] = __shfl_sync(0xffffffffu, g, b + u, kLanes);
        }
#pragma unroll
        for (int u = 0; u < kSlabBatch; ++u) acc = fma8(unpack(q[u]), w[u], acc);
      }
      j0 += kLanes;
      if (j0 >= k) break;
      route(t, j0 + l, id, g);
    }
    if (t >= T) continue;
    store8<8>(dx + t * ld_dx, c, H, acc + unpack(ar));
  }
}

template <typename TO>
cudaError_t launch_route_dx(const RouteGradArgs& a, cudaStream_t st) {
  constexpr int C = kSlabColumns;
  auto kern = route_dx_kernel<TO>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(kern, done);
  if (e != cudaSuccess) return e;
  const int slabs = (a.H + C - 1) / C, smem = (a.E + 1) * C * 2;
  const int per_sm = std::max(1, std::min(2048 / kSlabThreads, kNormSmem / smem));
  const int tokens = kSlabThreads / 32 * (256 / C);  // per CTA at a time
  const int parts = std::max(1, std::min(per_sm * sm_count() / slabs, (a.T + tokens - 1) / tokens));
  return launch_pdl(kern, dim3(slabs, parts), dim3(kSlabThreads), smem, st,
                    static_cast<const bf16_t*>(a.w_router.p), a.w_router.ld, a.ids, a.dlogits, a.T, a.k, a.E, a.H,
                    static_cast<TO*>(a.dx.p), a.dx.ld, static_cast<const TO*>(a.add.p), a.add.ld);
}

}  // namespace

size_t route_grad_ws_bytes(int T, int k, int E, int H) { return ws_layout(nullptr, T * k, E, H).bytes; }

cudaError_t launch_route_grad(const RouteGradArgs& a, cudaStream_t st) {
  const int R = a.T * a.k;
  const bool rows = a.dw_router.p != nullptr || a.dbias != nullptr, direct = a.T <= kDirectTokens;
  const int plan = rows && !direct;
  const Ws ws = ws_layout(a.ws, R, a.E, a.H);
  const int units = direct ? a.E : max_units(R, a.E), multi = direct ? 0 : max_multi(R, a.E);
  cudaError_t e = cudaSuccess;
  if (a.T > 0) {
    const int warps = kPlanThreads / 32, ctas = std::min((a.T + warps - 1) / warps, 4 * sm_count());
    e = launch_pdl(route_plan_kernel, dim3(ctas + plan), dim3(kPlanThreads), 0, st, a.dw, a.w, a.ids, a.offsets, a.T,
                   a.k, a.E, a.dlogits, ws.units, ws.multi, units, multi, plan, unit_for(R), a.status);
    if (e != cudaSuccess) return e;
  }
  if (a.dx.p != nullptr && a.T > 0) {
    const Rows none = {nullptr, 0, MOE_ROW_BF16};
    if (static_cast<int64_t>(R) * a.H >= kSlabElements && (a.E + 1) * kSlabColumns * 2 <= kNormSmem &&
        row_unit({a.w_router, a.dx, a.add}) == 8)
      e = a.dx.type == MOE_ROW_F32 ? launch_route_dx<float>(a, st) : launch_route_dx<bf16_t>(a, st);
    else
      e = launch_join(a.w_router, none, a.ids, a.dlogits, a.T, a.k, a.H, a.E, a.dx, a.add, nullptr, a.status, st);
    if (e != cudaSuccess) return e;
  }
  if (!rows) return cudaSuccess;
  const int pieces = a.dw_router.p != nullptr ? (a.H + 255) / 256 : 1;
  const int unit = row_unit({a.x, a.dw_router});
  auto go = [&](auto kern) {
    return launch_pdl(kern, dim3((units + kRowWarps - 1) / kRowWarps, pieces), dim3(kRowWarps * 32), 0, st, a.dlogits,
                      a.offsets, a.perm, static_cast<const bf16_t*>(a.x.p), a.x.ld, R, a.k, a.E, a.H, ws.units, units,
                      static_cast<float*>(a.dw_router.p), a.dw_router.ld, a.dbias, ws.rows, ws.bias, a.status);
  };
  if (direct)
    e = unit == 8   ? go(route_rows_kernel<8, true>)
        : unit == 2 ? go(route_rows_kernel<2, true>)
                    : go(route_rows_kernel<1, true>);
  else
    e = unit == 8   ? go(route_rows_kernel<8, false>)
        : unit == 2 ? go(route_rows_kernel<2, false>)
                    : go(route_rows_kernel<1, false>);
  if (e != cudaSuccess || multi == 0) return e;
  return launch_pdl(route_join_kernel, dim3(multi, (a.H + 1023) / 1024), dim3(256), 0, st, ws.multi, ws.rows, ws.bias,
                    a.H, static_cast<float*>(a.dw_router.p), a.dw_router.ld, a.dbias);
}

}  // namespace blk
}  // namespace moe
