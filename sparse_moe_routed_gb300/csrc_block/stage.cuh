// Rows staged through shared memory by asynchronous copies (the norms).
//
// A group of nt threads owns a row and thread `tid` its columns
//   col(h, i) = h * 8 nt + ((i / G) * nt + tid) * G + i % G,   i = 0..7
// for h = 0..NCH-1: G adjacent columns at a time, so that every access of a
// warp covers whole sectors (G = 4: 16 bytes of fp32, 8 of bf16 a lane; G = 2:
// rows that start on even columns; G = 1: any).  Each thread copies its own
// columns into its own places in shared memory and reads them back itself:
// copies of the rows ahead stay in flight while a row is worked on, cost no
// registers, and need no barrier, only the thread's own wait.
#pragma once

#include "rows.cuh"

namespace moe {
namespace blk {

// Bytes of one thread's eight columns of one array.
template <typename T>
constexpr int kSlot = 8 * static_cast<int>(sizeof(T));

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
  if (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES < 16 ? BYTES : 8) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most `left` of the thread's committed groups are in flight.
__device__ __forceinline__ void copies_wait(int left) {
  if (left >= 2)
    asm volatile("cp.async.wait_group 2;" ::: "memory");
  else if (left == 1)
    asm volatile("cp.async.wait_group 1;" ::: "memory");
  else
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

template <int G>
__device__ __forceinline__ int col0(int h, int i, int tid, int nt) {
  return (h * (8 / G) + i / G) * nt * G + tid * G + i % G;
}

// Thread's columns of a row into its places; columns past H become zero.
// The array's region holds NCH * nt * kSlot<T> bytes.
template <typename T, int G, int NCH>
__device__ __forceinline__ void stage_row(unsigned char* region, const T* row, int tid, int nt, int H) {
  constexpr int UB = G * static_cast<int>(sizeof(T));  // bytes of one unit of G columns
#pragma unroll
  for (int p = 0; p < NCH * 8 / G; ++p) {
    const int c = (p * nt + tid) * G;
    unsigned char* at = region + static_cast<size_t>(p * nt + tid) * UB;
    if (UB >= 4 && c + G <= H) {
      copy_async<(UB >= 4 ? UB : 4)>(static_cast<uint32_t>(__cvta_generic_to_shared(at)), row + c);
    } else {
#pragma unroll
      for (int i = 0; i < G; ++i) reinterpret_cast<T*>(at)[i] = c + i < H ? row[c + i] : T(0);
    }
  }
}

template <typename T, int G>
__device__ __forceinline__ void read_unit(const unsigned char* at, float* f) {
  if constexpr (sizeof(T) == 4) {
    if constexpr (G == 4) {
      const float4 v = *reinterpret_cast<const float4*>(at);
      f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
    } else if constexpr (G == 2) {
      const float2 v = *reinterpret_cast<const float2*>(at);
      f[0] = v.x, f[1] = v.y;
    } else {
      f[0] = *reinterpret_cast<const float*>(at);
    }
  } else {
    if constexpr (G == 4) {
      const uint2 v = *reinterpret_cast<const uint2*>(at);
      f[0] = __uint_as_float(v.x << 16), f[1] = __uint_as_float(v.x & 0xffff0000u);
      f[2] = __uint_as_float(v.y << 16), f[3] = __uint_as_float(v.y & 0xffff0000u);
    } else if constexpr (G == 2) {
      const uint32_t v = *reinterpret_cast<const uint32_t*>(at);
      f[0] = __uint_as_float(v << 16), f[1] = __uint_as_float(v & 0xffff0000u);
    } else {
      f[0] = bf16_to_f32(*reinterpret_cast<const bf16_t*>(at));
    }
  }
}

// Chunk h of the thread's columns from its places.
template <typename T, int G>
__device__ __forceinline__ void read_staged(const unsigned char* region, int h, int tid, int nt, float (&f)[8]) {
  constexpr int UB = G * static_cast<int>(sizeof(T));
#pragma unroll
  for (int p = 0; p < 8 / G; ++p)
    read_unit<T, G>(region + static_cast<size_t>((h * (8 / G) + p) * nt + tid) * UB, f + p * G);
}

// The same from global memory; columns past H read as zero.
template <typename T, int G>
__device__ __forceinline__ void read_global(const T* row, int h, int tid, int nt, int H, float (&f)[8]) {
#pragma unroll
  for (int p = 0; p < 8 / G; ++p) {
    const int c = ((h * (8 / G) + p) * nt + tid) * G;
    if (c + G <= H) {
      read_unit<T, G>(reinterpret_cast<const unsigned char*>(row + c), f + p * G);
    } else {
#pragma unroll
      for (int i = 0; i < G; ++i) f[p * G + i] = c + i < H ? as_f32(row[c + i]) : 0.f;
    }
  }
}

template <typename T, int G>
__device__ __forceinline__ void write_row(T* row, int h, int tid, int nt, int H, const float (&f)[8]) {
#pragma unroll
  for (int p = 0; p < 8 / G; ++p) {
    const int c = ((h * (8 / G) + p) * nt + tid) * G;
    if (c + G <= H) {
      if constexpr (sizeof(T) == 4) {
        if constexpr (G == 4)
          *reinterpret_cast<float4*>(row + c) = make_float4(f[p * G], f[p * G + 1], f[p * G + 2], f[p * G + 3]);
        else if constexpr (G == 2)
          *reinterpret_cast<float2*>(row + c) = make_float2(f[p * G], f[p * G + 1]);
        else
          row[c] = f[p];
      } else {
        if constexpr (G == 4)
          *reinterpret_cast<uint2*>(row + c) =
              make_uint2(pack2(f[p * G], f[p * G + 1]), pack2(f[p * G + 2], f[p * G + 3]));
        else if constexpr (G == 2)
          *reinterpret_cast<uint32_t*>(row + c) = pack2(f[p * G], f[p * G + 1]);
        else
          row[c] = f32_to_bf16(f[p]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < G; ++i)
        if (c + i < H) put(row + c + i, f[p * G + i]);
    }
  }
}

// Sum of v over the group's nt threads.  `buf` alternates between successive
// sums: a buffer is written again only after the barrier of the sum between.
__device__ __forceinline__ float group_sum(float v, float (*buf)[16], int& which, int tid, int nt, int group) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (nt == 32) return v;
  float* b = buf[which];
  which ^= 1;
  if ((tid & 31) == 0) b[tid >> 5] = v;
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(nt) : "memory");
  float s = 0.f;
  for (int i = 0; i < nt / 32; ++i) s += b[i];
  return s;
}

__device__ __forceinline__ float gain(const float* gamma, int c) { return gamma != nullptr ? 1.0f + gamma[c] : 1.0f; }

}  // namespace blk
}  // namespace moe
