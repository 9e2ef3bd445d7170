// Rows of activations into 8 bits and back (see q8.cuh for the format).
//
// Bound by HBM: save reads a row and writes a byte per element and a byte per
// 32; load reads those and writes a row, or the k rows of a token's routes, so
// that a token kept once is read once whatever k is.  One warp moves up to 1,024
// columns of one row in pieces of 256 (rows.cuh), all its loads in flight
// together; there is no barrier, and a group's largest value goes over the four
// lanes (sixteen, thirty-two for rows on even and odd elements) that hold it.
#include <algorithm>
#include <type_traits>

#include "launch.h"
#include "q8.cuh"
#include "rows.cuh"

namespace moe {
namespace blk {

namespace {

constexpr int kPieces = 4;  // of 256 columns, per warp
constexpr int kWarps = 8;   // per CTA

// Which row and which columns this warp has; false: none.
__device__ __forceinline__ bool my_part(int T, int parts, int64_t& t, int& base) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  t = i / parts;
  base = static_cast<int>(i - t * parts) * (kPieces * 256);
  return t < T;
}

// Eight bytes of a row of bytes: one access for U = 8, pairs for U = 2.
template <int U>
__device__ __forceinline__ void load_bytes(const uint8_t* row, const Cols<U>& c, int H, uint8_t (&b)[8]) {
  if (U == 8 && c.first + 8 <= H) {
    const uint2 v = *reinterpret_cast<const uint2*>(row + c.first);
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = static_cast<uint8_t>((i < 4 ? v.x : v.y) >> (8 * (i & 3)));
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const int a = c.at(i);
    if (U == 2 && a + 1 < H) {
      const uint32_t v = *reinterpret_cast<const uint16_t*>(row + a);
      b[i] = static_cast<uint8_t>(v);
      b[i + 1] = static_cast<uint8_t>(v >> 8);
    } else {
      b[i] = a < H ? row[a] : 0;
      b[i + 1] = c.at(i + 1) < H ? row[c.at(i + 1)] : 0;
    }
  }
}
template <int U>
__device__ __forceinline__ void store_bytes(uint8_t* row, const Cols<U>& c, int H, const uint32_t (&b)[8]) {
  if (U == 8 && c.first + 8 <= H) {
    *reinterpret_cast<uint2*>(row + c.first) =
        make_uint2(b[0] | b[1] << 8 | b[2] << 16 | b[3] << 24, b[4] | b[5] << 8 | b[6] << 16 | b[7] << 24);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const int a = c.at(i);
    if (U == 2 && a + 1 < H) {
      *reinterpret_cast<uint16_t*>(row + a) = static_cast<uint16_t>(b[i] | b[i + 1] << 8);
    } else {
      if (a < H) row[a] = static_cast<uint8_t>(b[i]);
      if (c.at(i + 1) < H) row[c.at(i + 1)] = static_cast<uint8_t>(b[i + 1]);
    }
  }
}

// Largest value of the group that each of the lane's units lies in.  U = 8: the
// lane's eight columns lie in one group, held by four lanes; U = 2: unit i of 16
// lanes is a group; U = 1: unit i of the warp.
template <int U>
__device__ __forceinline__ void group_max(uint32_t (&m)[8 / U]) {
#pragma unroll
  for (int i = 0; i < 8 / U; ++i) {
    if (U == 1) {
      m[i] = __reduce_max_sync(0xffffffffu, m[i]);
    } else {
#pragma unroll
      for (int d = 1; d < kGroup / U; d *= 2) m[i] = max(m[i], __shfl_xor_sync(0xffffffffu, m[i], d));
    }
  }
}

template <typename T_, int U>
__global__ void __launch_bounds__(kWarps * 32)
    save_kernel(const T_* __restrict__ x, int64_t ldx, int T, int H, int parts, uint8_t* q, int64_t ldq, uint8_t* exp,
                int64_t ld_exp) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  int64_t t;
  int base;
  if (!my_part(T, parts, t, base)) return;
  Raw8<T_> r[kPieces];
#pragma unroll
  for (int p = 0; p < kPieces; ++p)
    if (base + p * 256 < H) load8<U>(x + t * ldx, Cols<U>(base + p * 256, lane, 32), H, r[p]);
#pragma unroll
  for (int p = 0; p < kPieces; ++p) {
    if (base + p * 256 >= H) break;
    const Cols<U> c(base + p * 256, lane, 32);
    const V8 v = unpack(r[p]);
    uint32_t m[8 / U];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t a = __float_as_uint(el(v, i)) & 0x7fffffffu;
      m[i / U] = i % U == 0 ? a : max(m[i / U], a);
    }
    group_max<U>(m);
    uint32_t b[8];
#pragma unroll
    for (int i = 0; i < 8 / U; ++i) {
      const uint32_t e = exp_byte(m[i]);
      const float inv = inv_scale(e);
#pragma unroll
      for (int j = 0; j < U; ++j) b[i * U + j] = static_cast<uint32_t>(to_q8(el(v, i * U + j), inv)) & 255u;
      const int a = c.at(i * U);
      if (a % kGroup == 0 && a < H) exp[t * ld_exp + a / kGroup] = static_cast<uint8_t>(e);
    }
    store_bytes<U>(q + t * ldq, c, H, b);
  }
}

template <typename T_, int U>
__global__ void __launch_bounds__(kWarps * 32)
    load_kernel(const uint8_t* __restrict__ q, int64_t ldq, const uint8_t* __restrict__ exp, int64_t ld_exp, int T,
                int H, int parts, const int32_t* __restrict__ slot_of, const float* __restrict__ w, int k, int R,
                T_* out, int64_t ld_out, int32_t* status) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  int64_t t;
  int base;
  if (!my_part(T, parts, t, base)) return;
  int slot = -1;
  float weight = 1.f;
  if (slot_of != nullptr && lane < k) {
    slot = slot_of[t * k + lane];
    if (slot < -1 || slot >= R) {
      set_status(status, MOE_DEV_BAD_EXPERT);
      slot = -1;
    }
    if (w != nullptr) weight = w[t * k + lane];
  }
  uint8_t b[kPieces][8];
  uint32_t e[kPieces][8 / U];
#pragma unroll
  for (int p = 0; p < kPieces; ++p) {
    if (base + p * 256 >= H) break;
    const Cols<U> c(base + p * 256, lane, 32);
    load_bytes<U>(q + t * ldq, c, H, b[p]);
#pragma unroll
    for (int i = 0; i < 8 / U; ++i) e[p][i] = c.at(i * U) < H ? exp[t * ld_exp + c.at(i * U) / kGroup] : 0;
  }
  V8 v[kPieces];
#pragma unroll
  for (int p = 0; p < kPieces; ++p)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      el(v[p], i) = base + p * 256 < H ? static_cast<float>(static_cast<int8_t>(b[p][i])) * scale_of(e[p][i / U]) : 0.f;
  for (int j = 0; j < k; ++j) {
    const int64_t s = slot_of == nullptr ? t : __shfl_sync(0xffffffffu, slot, j);
    const float f = __shfl_sync(0xffffffffu, weight, j);
    if (s < 0) continue;
#pragma unroll
    for (int p = 0; p < kPieces; ++p)
      if (base + p * 256 < H)
        store8<U>(out + s * ld_out, Cols<U>(base + p * 256, lane, 32), H, w != nullptr ? v[p] * f : v[p]);
  }
}

// Rows of bytes on u-byte boundaries.
inline bool bytes_on(const Bytes& b, int u) { return b.ld % u == 0 && reinterpret_cast<uintptr_t>(b.p) % u == 0; }
inline int unit_of(const Rows& r, const Bytes& q) {
  for (int u : {8, 2})
    if (starts_on(r, u) && bytes_on(q, u)) return u;
  return 1;
}

template <typename F>
cudaError_t by_type(int type, int unit, F&& f) {
  auto g = [&](auto t) {
    if (unit == 8) return f(t, std::integral_constant<int, 8>());
    if (unit == 2) return f(t, std::integral_constant<int, 2>());
    return f(t, std::integral_constant<int, 1>());
  };
  return type == MOE_ROW_F32 ? g(float()) : g(bf16_t());
}

struct Grid {
  int parts;
  int64_t ctas;
  Grid(int T, int H)
      : parts((H + kPieces * 256 - 1) / (kPieces * 256)), ctas((static_cast<int64_t>(T) * parts + kWarps - 1) / kWarps) {}
};

}  // namespace

cudaError_t launch_checkpoint_save(const Rows& x, int T, int H, const Bytes& q, const Bytes& exp, cudaStream_t st) {
  const Grid g(T, H);
  return by_type(x.type, unit_of(x, q), [&](auto t, auto u) {
    using T_ = decltype(t);
    return launch_pdl(save_kernel<T_, decltype(u)::value>, dim3(static_cast<unsigned>(g.ctas)), dim3(kWarps * 32), 0,
                      st, static_cast<const T_*>(x.p), x.ld, T, H, g.parts, q.p, q.ld, exp.p, exp.ld);
  });
}

cudaError_t launch_checkpoint_load(const Bytes& q, const Bytes& exp, int T, int H, const int32_t* slot_of,
                                   const float* w, int k, int R, const Rows& out, int32_t* status, cudaStream_t st) {
  const Grid g(T, H);
  return by_type(out.type, unit_of(out, q), [&](auto t, auto u) {
    using T_ = decltype(t);
    return launch_pdl(load_kernel<T_, decltype(u)::value>, dim3(static_cast<unsigned>(g.ctas)), dim3(kWarps * 32), 0,
                      st, q.p, q.ld, exp.p, exp.ld, T, H, g.parts, slot_of, w, k, R, static_cast<T_*>(out.p), out.ld,
                      status);
  });
}

}  // namespace blk
}  // namespace moe
