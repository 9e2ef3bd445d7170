// Rows of fp32 or bf16 elements, moved eight elements per lane.
//
// A row is cut into pieces of 8 elements per thread, in units of U adjacent
// elements.  U = 8, where all rows start on 8-element boundaries: one 16 byte
// access for bf16, one 32 byte access for fp32, so that bf16 and fp32 rows of
// one call are indexed alike and every access fills whole 32 byte sectors.
// U = 2, where they start on even elements, and U = 1: the units are n threads
// apart, so that a warp's accesses are adjacent.  A row's last piece and its
// last unit may be partial.
#pragma once

#include <stdint.h>

#include "../csrc/common.cuh"

namespace moe {
namespace blk {

using bf16_t = uint16_t;

// Eight raw elements as they sit in registers.
template <typename T>
struct Raw8;
template <>
struct Raw8<float> {
  float v[8];
};
template <>
struct Raw8<bf16_t> {
  uint32_t v[4];
};

// Eight columns as four pairs: two fp32 operations per instruction.
struct V8 {
  float2 v[4];
};
__device__ __forceinline__ float& el(V8& f, int i) { return i & 1 ? f.v[i / 2].y : f.v[i / 2].x; }
__device__ __forceinline__ float el(const V8& f, int i) { return i & 1 ? f.v[i / 2].y : f.v[i / 2].x; }
__device__ __forceinline__ float2 splat(float a) { return make_float2(a, a); }
__device__ __forceinline__ V8 operator*(const V8& a, const V8& b) {
  V8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.v[i] = __fmul2_rn(a.v[i], b.v[i]);
  return r;
}
__device__ __forceinline__ V8 operator*(const V8& a, float b) {
  V8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.v[i] = __fmul2_rn(a.v[i], splat(b));
  return r;
}
__device__ __forceinline__ V8 fma8(const V8& a, const V8& b, const V8& c) {
  V8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.v[i] = __ffma2_rn(a.v[i], b.v[i], c.v[i]);
  return r;
}
__device__ __forceinline__ V8 fma8(const V8& a, float b, const V8& c) {
  V8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.v[i] = __ffma2_rn(a.v[i], splat(b), c.v[i]);
  return r;
}
__device__ __forceinline__ V8 operator+(const V8& a, const V8& b) {
  V8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.v[i] = __fadd2_rn(a.v[i], b.v[i]);
  return r;
}
__device__ __forceinline__ V8 zero8() {
  V8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.v[i] = splat(0.f);
  return r;
}
// s += sum a b
__device__ __forceinline__ void dot8(const V8& a, const V8& b, float2& s) {
#pragma unroll
  for (int i = 0; i < 4; ++i) s = __ffma2_rn(a.v[i], b.v[i], s);
}

__device__ __forceinline__ float2 widen(uint32_t two) {
  return make_float2(__uint_as_float(two << 16), __uint_as_float(two & 0xffff0000u));
}

__device__ __forceinline__ V8 unpack(const Raw8<float>& r) {
  V8 f;
#pragma unroll
  for (int i = 0; i < 4; ++i) f.v[i] = make_float2(r.v[2 * i], r.v[2 * i + 1]);
  return f;
}
__device__ __forceinline__ V8 unpack(const Raw8<bf16_t>& r) {
  V8 f;
#pragma unroll
  for (int i = 0; i < 4; ++i) f.v[i] = widen(r.v[i]);
  return f;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;  // round to nearest even, NaN stays NaN
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void pack(const V8& f, Raw8<float>& r) {
#pragma unroll
  for (int i = 0; i < 4; ++i) r.v[2 * i] = f.v[i].x, r.v[2 * i + 1] = f.v[i].y;
}
__device__ __forceinline__ void pack(const V8& f, Raw8<bf16_t>& r) {
#pragma unroll
  for (int i = 0; i < 4; ++i) r.v[i] = pack2(f.v[i].x, f.v[i].y);
}

// Whole pieces.  Plain (coherent) loads: an output may be its own input.
__device__ __forceinline__ void load_vec(const float* p, Raw8<float>& r) {
  asm volatile("ld.global.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(r.v[0]), "=f"(r.v[1]), "=f"(r.v[2]), "=f"(r.v[3]), "=f"(r.v[4]), "=f"(r.v[5]), "=f"(r.v[6]),
                 "=f"(r.v[7])
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void load_vec(const bf16_t* p, Raw8<bf16_t>& r) {
  asm volatile("ld.global.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.v[0]), "=r"(r.v[1]), "=r"(r.v[2]), "=r"(r.v[3])
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void store_vec(float* p, const Raw8<float>& r) {
  asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(r.v[0]), "f"(r.v[1]), "f"(r.v[2]),
               "f"(r.v[3]), "f"(r.v[4]), "f"(r.v[5]), "f"(r.v[6]), "f"(r.v[7])
               : "memory");
}
__device__ __forceinline__ void store_vec(bf16_t* p, const Raw8<bf16_t>& r) {
  asm volatile("st.global.v4.b32 [%0], {%1,%2,%3,%4};" ::"l"(p), "r"(r.v[0]), "r"(r.v[1]), "r"(r.v[2]), "r"(r.v[3])
               : "memory");
}

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(bf16_t* p, float v) { *p = f32_to_bf16(v); }

__device__ __forceinline__ void raw_set(Raw8<float>& r, int i, float v) { r.v[i] = v; }
__device__ __forceinline__ void raw_set(Raw8<bf16_t>& r, int i, bf16_t v) {
  if (i & 1)
    r.v[i >> 1] |= static_cast<uint32_t>(v) << 16;
  else
    r.v[i >> 1] = v;
}
template <typename T>
__device__ __forceinline__ void raw_zero(Raw8<T>& r) {
#pragma unroll
  for (unsigned i = 0; i < sizeof(r.v) / sizeof(r.v[0]); ++i) r.v[i] = 0;
}

// Which columns thread `tid` of `n` holds of the piece that starts at column
// `base` and spans 8 n columns.
template <int U>
struct Cols {
  int first;  // of the thread's first unit
  int step;   // from unit to unit
  __device__ __forceinline__ Cols(int base, int tid, int n) : first(base + tid * U), step(n * U) {}
  __device__ __forceinline__ int at(int i) const { return first + i / U * step + i % U; }
};

// Two adjacent elements of a row that starts on an even one.
__device__ __forceinline__ void load_pair(const float* p, int i, Raw8<float>& r) {
  asm volatile("ld.global.v2.f32 {%0,%1}, [%2];" : "=f"(r.v[i]), "=f"(r.v[i + 1]) : "l"(p) : "memory");
}
__device__ __forceinline__ void load_pair(const bf16_t* p, int i, Raw8<bf16_t>& r) {
  asm volatile("ld.global.b32 %0, [%1];" : "=r"(r.v[i / 2]) : "l"(p) : "memory");
}
__device__ __forceinline__ void store_pair(float* p, float2 v) { *reinterpret_cast<float2*>(p) = v; }
__device__ __forceinline__ void store_pair(bf16_t* p, float2 v) { *reinterpret_cast<uint32_t*>(p) = pack2(v.x, v.y); }

// Elements past column H read as zero.
template <int U, typename T>
__device__ __forceinline__ void load8(const T* row, const Cols<U>& c, int H, Raw8<T>& r) {
  if (U == 8 && c.first + 8 <= H) {
    load_vec(row + c.first, r);
    return;
  }
  raw_zero(r);
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const int a = c.at(i);
    if (U == 2 && a + 1 < H) {
      load_pair(row + a, i, r);
    } else {
      if (a < H) raw_set(r, i, row[a]);
      if (c.at(i + 1) < H) raw_set(r, i + 1, row[c.at(i + 1)]);
    }
  }
}
template <int U, typename T>
__device__ __forceinline__ void store8(T* row, const Cols<U>& c, int H, const V8& f) {
  if (U == 8 && c.first + 8 <= H) {
    Raw8<T> r;
    pack(f, r);
    store_vec(row + c.first, r);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const int a = c.at(i);
    if (U == 2 && a + 1 < H) {
      store_pair(row + a, f.v[i / 2]);
    } else {
      if (a < H) put(row + a, el(f, i));
      if (c.at(i + 1) < H) put(row + c.at(i + 1), el(f, i + 1));
    }
  }
}

}  // namespace blk
}  // namespace moe
