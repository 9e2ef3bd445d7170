// Rows staged through shared memory by asynchronous copies (the norms).
//
// A group of nt threads owns a row and thread `tid` its columns
//   col(h, i) = h * 8 nt + ((i / G) * nt + tid) * G + i % G,   i = 0..7
// for h = 0..NCH-1: G adjacent columns at a time (G divides H), so that every
// access of a warp covers whole sectors (G = 4: 16 bytes of fp32, 8 of bf16 a
// lane; G = 2: even widths; G = 1: any) and no unit of G is partial.  Each
// thread copies its own columns into its own places in shared memory and reads
// them back itself: the copy of the row ahead stays in flight while a row is
// worked on, costs no registers, and needs no barrier, only the thread's own
// wait.
#pragma once

#include "launch.h"
#include "rows.cuh"

namespace moe {
namespace blk {

// Bytes of one thread's eight columns of one array.
template <typename T>
constexpr int kSlot = 8 * static_cast<int>(sizeof(T));

// BYTES from src to shared memory; `have` 0: zeros instead, src is not read.
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, int have) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(have) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(dst), "l"(src), "r"(have), "n"(BYTES)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits for all of the thread's copies.
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

template <int G>
__device__ __forceinline__ int col0(int h, int i, int tid, int nt) {
  return (h * (8 / G) + i / G) * nt * G + tid * G + i % G;
}

// Rows that start on any element (G = 1) would take many narrow copies that
// way, and bf16 ones none at all (a copy has four bytes at least).  Their group
// copies the aligned 16-byte chunks that hold the row instead, into the
// operand's region of shared memory from its start on, and after a barrier a
// thread reads its columns from there, as many bytes on as the row starts
// behind its first chunk.  What the first chunk holds in front of the row is
// read, but not used; a chunk that holds one byte of an allocation lies inside
// it.
template <int G>
constexpr bool kByChunks = G == 1;

// Bytes of one operand's row in a stage.
template <typename T, int G, int NCH>
__device__ __forceinline__ int region(int nt) {
  return NCH * nt * kSlot<T> + (kByChunks<G> ? 16 : 0);
}

// A thread's share of a row into the operand's region, columns past H as
// zeros.  src: the thread's first column of the row; at: its first place.
template <typename T, int G, int NCH>
__device__ __forceinline__ void stage_row(unsigned char* at, const T* src, int tid, int nt, int H) {
  constexpr int UB = G * static_cast<int>(sizeof(T));  // bytes of one unit of G columns
  const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(at));
  if constexpr (kByChunks<G>) {
    const uintptr_t row = reinterpret_cast<uintptr_t>(src - tid * G), from = row & ~static_cast<uintptr_t>(15);
    const int end = static_cast<int>(row - from) + H * static_cast<int>(sizeof(T));  // of the row in its region
    // two chunks of zeros more: the row before may have ended that far on
    const int chunks = min(NCH * nt * kSlot<T> / 16 + 1, (end + 15) / 16 + 2);
    for (int w = tid; w < chunks; w += nt) {
      const int have = max(0, min(16, end - 16 * w));
      copy_async<16>(to - tid * UB + 16 * w, reinterpret_cast<const void*>(have > 0 ? from + 16 * w : from), have);
    }
  } else {
#pragma unroll
    for (int p = 0; p < NCH * 8 / G; ++p)
      copy_async<UB>(to + p * nt * UB, src + p * nt * G, (p * nt + tid) * G < H ? UB : 0);
  }
}

// Unit p of G columns.
template <typename T, int G>
__device__ __forceinline__ void read_unit(const unsigned char* at, int p, V8& f) {
  if constexpr (sizeof(T) == 4) {
    if constexpr (G == 4) {
      const float4 v = *reinterpret_cast<const float4*>(at);
      f.v[2 * p] = make_float2(v.x, v.y);
      f.v[2 * p + 1] = make_float2(v.z, v.w);
    } else if constexpr (G == 2) {
      f.v[p] = *reinterpret_cast<const float2*>(at);
    } else {
      el(f, p) = *reinterpret_cast<const float*>(at);
    }
  } else {
    if constexpr (G == 4) {
      const uint2 v = *reinterpret_cast<const uint2*>(at);
      f.v[2 * p] = widen(v.x);
      f.v[2 * p + 1] = widen(v.y);
    } else if constexpr (G == 2) {
      f.v[p] = widen(*reinterpret_cast<const uint32_t*>(at));
    } else {
      el(f, p) = bf16_to_f32(*reinterpret_cast<const bf16_t*>(at));
    }
  }
}

// Chunk h of the thread's columns; at: its first place, row: where the row
// starts in global memory (by chunks only; null: in the region's first byte).
template <typename T, int G>
__device__ __forceinline__ void read_staged(const unsigned char* at, const T* row, int h, int nt, V8& f) {
  constexpr int UB = G * static_cast<int>(sizeof(T));
  if (kByChunks<G>) at += reinterpret_cast<uintptr_t>(row) & 15;
#pragma unroll
  for (int p = 0; p < 8 / G; ++p) read_unit<T, G>(at + (h * (8 / G) + p) * nt * UB, p, f);
}

// The group's threads meet (staging by chunks).
__device__ __forceinline__ void group_sync(int nt, int group) {
  if (nt == 32)
    __syncwarp();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(nt) : "memory");
}

// The same from global memory; columns past H read as zero.
template <typename T, int G>
__device__ __forceinline__ void read_global(const T* row, int h, int tid, int nt, int H, V8& f) {
#pragma unroll
  for (int p = 0; p < 8 / G; ++p) {
    const int c = ((h * (8 / G) + p) * nt + tid) * G;
#pragma unroll
    for (int i = 0; i < G; ++i) el(f, p * G + i) = 0.f;
    if (c < H) read_unit<T, G>(reinterpret_cast<const unsigned char*>(row + c), p, f);
  }
}

// dst: the thread's first column of the row.
template <typename T, int G>
__device__ __forceinline__ void write_row(T* dst, int h, int tid, int nt, int H, const V8& f) {
#pragma unroll
  for (int p = 0; p < 8 / G; ++p) {
    const int at = (h * (8 / G) + p) * nt * G;
    if (at + tid * G >= H) continue;
    if constexpr (sizeof(T) == 4) {
      if constexpr (G == 4)
        *reinterpret_cast<float4*>(dst + at) =
            make_float4(f.v[2 * p].x, f.v[2 * p].y, f.v[2 * p + 1].x, f.v[2 * p + 1].y);
      else if constexpr (G == 2)
        *reinterpret_cast<float2*>(dst + at) = f.v[p];
      else
        dst[at] = el(f, p);
    } else {
      if constexpr (G == 4)
        *reinterpret_cast<uint2*>(dst + at) =
            make_uint2(pack2(f.v[2 * p].x, f.v[2 * p].y), pack2(f.v[2 * p + 1].x, f.v[2 * p + 1].y));
      else if constexpr (G == 2)
        *reinterpret_cast<uint32_t*>(dst + at) = pack2(f.v[p].x, f.v[p].y);
      else
        dst[at] = f32_to_bf16(el(f, p));
    }
  }
}

// The thread's first column of row `row`; null rows stay null.
template <typename T>
__device__ __forceinline__ T* first_column(const Rows& r, int64_t row, int col) {
  return r.p == nullptr ? nullptr : static_cast<T*>(r.p) + row * r.ld + col;
}
// Moves p by a launch constant (bytes), which the instruction itself can hold.
template <typename T>
__device__ __forceinline__ void advance(T*& p, int64_t bytes) {
  p = reinterpret_cast<T*>(reinterpret_cast<uintptr_t>(p) + bytes);
}

// Sum of v over the group's nt threads, four warps' sums to a read.  `buf`
// (zeros behind the group's warps) alternates between successive sums: a
// buffer is written again only after the barrier of the sum between.
__device__ __forceinline__ float group_sum(float v, float (*buf)[16], int& which, int tid, int nt, int group) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (nt == 32) return v;
  float* b = buf[which];
  which ^= 1;
  if ((tid & 31) == 0) b[tid >> 5] = v;
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(nt) : "memory");
  float s = 0.f;
  for (int i = 0; i < nt; i += 128) {
    const float4 w = *reinterpret_cast<const float4*>(b + i / 32);
    s += (w.x + w.y) + (w.z + w.w);
  }
  return s;
}
// Zeros the buffers of every group's sums and the rows' places; the CTA's
// threads call it together.
__device__ __forceinline__ void stage_init(float (*buf)[2][16], unsigned char* smem, int bytes) {
  for (int i = threadIdx.x; i < 15 * 2 * 16; i += blockDim.x) (&buf[0][0][0])[i] = 0.f;
  for (int i = threadIdx.x * 16; i < bytes; i += blockDim.x * 16)
    *reinterpret_cast<uint4*>(smem + i) = make_uint4(0, 0, 0, 0);
  __syncthreads();
}

__device__ __forceinline__ float gain(const float* gamma, int c) { return gamma != nullptr ? 1.0f + gamma[c] : 1.0f; }

}  // namespace blk
}  // namespace moe
